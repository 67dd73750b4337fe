"""The example layer end to end: outputs and gradients against float64 autograd
with the same routing, training that lowers the loss, 8-bit serving."""

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import ragged_moe_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def _reference(layer, x, ids, dout):
    """float64, differentiated by torch; the choice of experts is given."""
    w = [t.double().requires_grad_() for t in (layer.router, layer.w1, layer.w2)]
    xd = x.double().requires_grad_()
    live = ids >= 0
    logits = (xd @ w[0].T).gather(1, ids.clamp(min=0).long())
    weights = torch.softmax(torch.where(live, logits, -1e30), 1) * live
    out = torch.zeros_like(xd)
    for e in range(len(layer.router)):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            gate, up = (xd[t] @ w[1][e].T).chunk(2, dim=1)
            out = out.index_add(0, t, weights[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ w[2][e].T))
    out.backward(dout.double())
    return out.detach(), xd.grad, [t.grad for t in w]


@pytest.mark.parametrize("tokens,experts,hidden,ffn,top_k,masked", [
    (1, 8, 128, 64, 2, False), (77, 5, 200, 72, 3, True), (1000, 16, 512, 256, 4, False)])
def test_layer(tokens, experts, hidden, ffn, top_k, masked):
    layer = ex.Layer.random(experts, hidden, ffn, top_k).bf16()
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((tokens, hidden), generator=gen, device="cuda").bfloat16()
    dout = torch.randn((tokens, hidden), generator=gen, device="cuda").bfloat16()
    mask = torch.rand(tokens, generator=gen, device="cuda") < 0.8 if masked else None
    out, saved = ex.forward(layer, x, mask)
    dx, grad = ex.backward(layer, saved, dout)
    ref, rdx, rgrad = _reference(layer, x, saved[2].ids, dout)
    # at most 8 roundings to bf16 lie on any path (h, a, y, out; dy, da, dh, dx or
    # dlogits), half a step (2^-8) each, relative to the norm
    tol = 8 * 2.0 ** -8
    near = lambda a, b: float((a.double() - b).norm()) <= tol * float(b.norm())  # noqa: E731
    assert near(out, ref) and near(dx, rdx)
    for a, b in zip((grad.router, grad.w1, grad.w2), rgrad):
        assert near(a, b)
    # 8-bit: codes are off by half a step of amax / 127 each; for normal values amax is
    # about 3.5 standard deviations, so about 0.8 % of the norm for each of four
    # quantized operands, beside the roundings above
    q = ex.serve(ex.Int8Layer.of(layer), x, mask)
    assert float((q.double() - ref).norm()) <= (tol + 4 * 0.016) * float(ref.norm())


def test_training_lowers_the_loss():
    layer, losses = ex.train(12, tokens=600, experts=8, hidden=256, ffn=256)
    assert all(bool(torch.isfinite(t).all()) for t in (layer.router, layer.w1, layer.w2))
    assert losses[-1] < 0.8 * losses[0]
    x = torch.randn((33, 256), generator=torch.Generator("cuda").manual_seed(9), device="cuda").bfloat16()
    out, saved = ex.forward(layer.bf16(), x)
    assert int(saved[2].m_splits.sum()) == 66
    got = ex.serve(ex.Int8Layer.of(layer.bf16()), x)
    assert float((got.float() - out.float()).norm()) < 0.1 * float(out.float().norm())
