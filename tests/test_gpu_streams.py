"""Calls on a stream that is not torch's current one."""

import pytest
import torch

import moe_expert_grouped_group_amd as mx

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _normal(shape, seed, dtype=BF):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def test_no_block_of_the_current_stream(monkeypatch):
    """A workspace that a call on the current stream has just dropped is not handed
    to a call on another stream."""
    x, w = _normal((600, 520), 1), _normal((4, 264, 520), 2)
    dy, ms = _normal((600, 264), 3), torch.tensor([300, 0, 41, 259], device="cuda")
    real, blocks = torch.empty, []

    def empty(*args, **kw):
        t = real(*args, **kw)
        blocks.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()))
        return t

    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", empty)
    first = [mx.ragged_gemm("NN", dy, w, ms), mx.ragged_gemm("TN", dy, x, ms)]
    dropped, blocks[:] = list(blocks), []
    s = torch.cuda.Stream()
    again = [mx.ragged_gemm("NN", dy, w, ms, stream=s), mx.ragged_gemm("TN", dy, x, ms, stream=s)]
    assert len(dropped) == 4 and len(blocks) == 4
    for lo, hi in blocks:
        assert all(hi <= a or b <= lo for a, b in dropped)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_quantizer_routing_and_join_on_another_stream():
    t, e, k, h = 700, 32, 4, 264
    z, x, dout = _normal((t, e), 1, torch.float32), _normal((t, h), 2), _normal((t, h), 3)
    w, y = _normal((e, 72, h), 4), _normal((t * k, h), 5)
    mask = torch.rand(t, generator=torch.Generator("cuda").manual_seed(6), device="cuda") < 0.9

    def calls(stream):
        wq, ws = mx.quantize_int8(w.view(-1, h), stream=stream)
        q, sc = mx.quantize_int8(x, stream=stream)
        r = mx.moe_route(z, k, token_mask=mask, stream=stream)
        c = mx.ragged_gemm_int8(q, sc, wq.view(w.shape), ws.view(e, 72), r.m_splits, row_index=r.row_token,
                                out=out, stream=stream)
        o = mx.moe_combine(y, r.row_pos, r.weights, stream=stream)
        dy, dw = mx.moe_combine_bwd(dout, y, r.row_pos, r.weights, out=(held, None), stream=stream)
        dz = mx.moe_route_bwd(z, r, dw, stream=stream)
        return [wq, ws, q, sc, r.ids, r.weights, r.m_splits, r.row_token, r.row_pos, c, o, dy, dw, dz]

    out, held = torch.zeros((t * k, 72), dtype=BF, device="cuda"), torch.zeros_like(y)
    first = [v.clone() for v in calls(None)]
    out.zero_()
    held.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = calls(s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
