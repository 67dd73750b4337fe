"""The gated, 8-bit floating-point and norm operators together, as a block uses them: the
example's blocks against float64 autograd, 8-bit serving, graphs, and other streams."""

import os
import sys

import pytest
import torch

import moe_expert_grouped_group_amd as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import ragged_moe_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _draw(shape, seed, dtype=F32, std=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _normed(v, w):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w


def _layer64(w, x, ids):
    """A layer in float64; the choice of experts is given."""
    router, w1, w2 = w
    live = ids >= 0
    logits = torch.matmul(x, router.T.contiguous()).gather(1, ids.clamp(min=0).long())
    weights = torch.softmax(torch.where(live, logits, -1e30), 1) * live
    out = torch.zeros_like(x)
    for e in range(len(router)):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            gate, up = torch.matmul(x[t], w1[e].T.contiguous()).chunk(2, dim=1)
            y = torch.matmul(gate * torch.sigmoid(gate) * up, w2[e].T.contiguous())
            out = out.index_add(0, t, weights[t, j, None] * y)
    return out


@pytest.mark.parametrize("tokens,experts,hidden,ffn,top_k,masked", [
    (1, 8, 128, 64, 2, False), (77, 5, 200, 72, 3, True), (700, 16, 512, 256, 4, False)])
def test_blocks(tokens, experts, hidden, ffn, top_k, masked):
    """Two blocks in a residual stream, forward and all gradients."""
    blocks = [ex.Block(ex.Layer.random(experts, hidden, ffn, top_k, seed=s).bf16(),
                       1 + 0.2 * _draw((hidden,), 10 + s), 1 + 0.2 * _draw((hidden,), 20 + s), 0.75) for s in (1, 2)]
    first = 1 + 0.2 * _draw((hidden,), 30)
    x, dy = _draw((tokens, hidden), 5, BF), _draw((tokens, hidden), 6, BF)
    mask = torch.rand(tokens, generator=torch.Generator("cuda").manual_seed(7), device="cuda") < 0.8 if masked else None
    y, kept = ex.blocks_forward(blocks, first, x, mask)
    dx, dfirst, grads = ex.blocks_backward(blocks, first, kept, dy)

    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    x64, first64 = leaf(x), leaf(first)
    w = [[leaf(t) for t in (b.layer.router, b.layer.w1, b.layer.w2, b.post, b.next)] for b in blocks]
    stream, norm = x64, _normed(x64, first64)
    for b, ws, (saved, _, _) in zip(blocks, w, kept[1:]):
        stream = b.scale * stream + _normed(_layer64(ws[:3], norm, saved[2].ids), ws[3])
        norm = _normed(stream, ws[4])
    norm.backward(dy.double())
    # Each block rounds to bf16 at most 8 times on any path through its layer (h, a, y, out; dy, da, dh,
    # dx or dlogits) and at most 4 times around it (stream, y; dstream, df), half a step (2^-8) each,
    # relative to the norm; two blocks and the first norm
    tol = (2 * 12 + 2) * 2.0 ** -8
    near = lambda a, b: float((a.double() - b).norm()) <= tol * float(b.norm())  # noqa: E731
    assert near(y, norm.detach()) and near(dx, x64.grad) and near(dfirst, first64.grad)
    for grad, ws in zip(grads, w):
        for got, want in zip((grad.layer.router, grad.layer.w1, grad.layer.w2, grad.post, grad.next), ws):
            assert near(got, want.grad)


@pytest.mark.parametrize("tokens,experts,hidden,ffn,top_k,masked", [
    (1, 8, 128, 64, 2, False), (77, 5, 200, 72, 3, True), (1000, 16, 512, 256, 4, False)])
def test_serving_in_fp8(tokens, experts, hidden, ffn, top_k, masked):
    layer = ex.Layer.random(experts, hidden, ffn, top_k).bf16()
    x = _draw((tokens, hidden), 5, BF)
    mask = torch.rand(tokens, generator=torch.Generator("cuda").manual_seed(7), device="cuda") < 0.8 if masked else None
    out, saved = ex.forward(layer, x, mask)
    want = _layer64([t.double() for t in (layer.router, layer.w1, layer.w2)], x.double(), saved[2].ids)
    got = ex.serve_fp8(ex.Fp8Layer.of(layer), x, mask)
    # e4m3 codes are off by at most 2^-4 of a value each, in four operands; half a step of bf16 in four results
    assert float((got.double() - want).norm()) <= (4 * 2.0 ** -4 + 4 * 2.0 ** -8) * float(want.norm())
    assert torch.isfinite(got).all()


def test_decode_step_in_a_graph():
    """Norm, router, gated experts, join and norm of a decode step in one graph, and its 8-bit form,
    replayed on new tokens with eager work between."""
    t, experts, hidden, ffn, top_k = 6, 16, 512, 256, 2
    layer = ex.Layer.random(experts, hidden, ffn, top_k).bf16()
    low = ex.Fp8Layer.of(layer)
    block = ex.Block(layer, 1 + 0.2 * _draw((hidden,), 1), 1 + 0.2 * _draw((hidden,), 2))
    first = 1 + 0.2 * _draw((hidden,), 3)
    x = _draw((t, hidden), 4, BF)
    ones = ex._all(t)

    def step(experts_of):
        stream, y = mx.residual_norm(x, pre_weight=first)
        logits = mx.ragged_gemm("NT", y, layer.router[None], ones, out_dtype=F32)
        route = mx.moe_route(logits, top_k)
        out = mx.moe_combine(experts_of(y, route), route.row_pos, route.weights)
        return mx.residual_norm(stream, out, post_weight=block.post, pre_weight=block.next)

    def gated(y, route):
        _, a = mx.ragged_gemm_swiglu(y, layer.w1, route.m_splits, row_index=route.row_token, want_h=False)
        return mx.ragged_gemm("NT", a, layer.w2, route.m_splits)

    def fp8(y, route):
        h = mx.ragged_gemm_fp8(*mx.quantize_fp8(y), low.w1, low.s1, route.m_splits, row_index=route.row_token)
        return mx.ragged_gemm_fp8(*mx.quantize_fp8(mx.swiglu_fwd(h)), low.w2, low.s2, route.m_splits)

    for experts_of in (gated, fp8):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(experts_of)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step(experts_of)
        for seed in range(3):
            x.copy_(_draw((t, hidden), 40 + seed, BF))
            graph.replay()
            got = [v.clone() for v in captured]
            want = step(experts_of)
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def _every_call(stream, x, dy, ms, index, w1, w2, wq, first, post, gate):
    h, a = mx.ragged_gemm_swiglu(x, w1, ms, row_index=index, stream=stream)
    _, only = mx.ragged_gemm_swiglu(x, w1, ms, row_index=index, want_h=False, stream=stream)
    dh, again = mx.ragged_gemm_swiglu_bwd(dy, w2, h, ms, stream=stream)
    codes = mx.quantize_fp8_weight(wq, stream=stream)
    q = mx.quantize_fp8(x, stream=stream)
    y = mx.ragged_gemm_fp8(*q, *codes, ms, row_index=index, stream=stream)
    y32 = mx.ragged_gemm_fp8(*q, *codes, ms, row_index=index, out_dtype=F32, stream=stream)
    kw = dict(gate=gate, post_weight=post, pre_weight=first, stream=stream)
    r, n = mx.residual_norm(x, dy[:len(x)], **kw)
    g = mx.residual_norm_bwd(n, r, r, dy[:len(x)], **kw)
    bytes_of = lambda t: t.view(torch.uint8)  # noqa: E731
    return [h, a, only, dh, again, bytes_of(codes[0]), codes[1], bytes_of(q[0]), q[1], y, y32, r, n, g.x, g.f, g.gate,
            g.post_weight, g.pre_weight]


def _operands(seed, rows=700, tokens=400, k=264, f=136):
    splits = [300, 0, 41, rows - 341]
    index = torch.randint(0, tokens, (rows,), generator=torch.Generator().manual_seed(seed)).int().cuda()
    return (_draw((tokens, k), seed, BF), _draw((rows, k), seed + 1, BF), torch.tensor(splits, device="cuda"), index,
            _draw((4, 2 * f, k), seed + 2, BF, 0.06), _draw((4, k, f), seed + 3, BF, 0.08),
            _draw((4, 200, k), seed + 4, BF), 1 + 0.2 * _draw((k,), seed + 5), 1 + 0.2 * _draw((k,), seed + 6),
            torch.sigmoid(_draw((tokens,), seed + 7)))


def test_calls_on_another_stream():
    args = _operands(1)
    first = [v.clone() for v in _every_call(None, *args)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = _every_call(s, *args)
    torch.cuda.current_stream().wait_stream(s)
    for i, (a, b) in enumerate(zip(first, again)):
        assert torch.equal(a, b), i


def test_two_streams_at_once():
    """Calls that run side by side, each on its own data, buffers and workspaces."""
    sets = [_operands(1), _operands(50)]
    want = [[v.clone() for v in _every_call(None, *s)] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [_every_call(st, *s) for st, s in zip(streams, sets)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for i, (u, v) in enumerate(zip(a, b)):
                assert torch.equal(u, v), i
