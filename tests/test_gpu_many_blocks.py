"""Sizes whose workgroups hold 2^32 threads or more, which one launch does not take:
the last rows, tokens and columns are where later launches work."""

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from gpu_util import log

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _pattern(n, seed, dtype=BF):
    """n values, a random run again and again."""
    gen = torch.Generator("cuda").manual_seed(seed)
    run = torch.randn(min(n, (1 << 20) + 7), generator=gen, device="cuda").to(dtype)
    return run.repeat(-(-n // run.numel()))[:n]


def _equal(got, want, step=1 << 27):
    """want(lo, hi) is the slice [lo, hi) of the result."""
    for lo in range(0, len(got), step):
        hi = min(lo + step, len(got))
        assert torch.equal(got[lo:hi], want(lo, hi)), (lo, hi)


def test_quantize_int8():
    t = (1 << 26) + 5                   # 64 threads a row
    log(f"quantize_int8 {t} x 3")
    x = _pattern(3 * t, 1).view(t, 3)
    q, s = mx.quantize_int8(x)

    def codes(lo, hi):
        v = x[lo:hi].double()
        scale = (v.abs().amax(1) / 127).float()
        return torch.round(v / scale.double()[:, None]).to(torch.int8)

    _equal(s, lambda lo, hi: (x[lo:hi].double().abs().amax(1) / 127).float(), 1 << 24)
    _equal(q, codes, 1 << 24)


def test_combine_and_its_gradient():
    t = (1 << 26) + 5                   # 4 tokens a workgroup of 256
    log(f"moe_combine {t} x 1")
    y = torch.randn((7, 1), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF)
    pos = (torch.arange(t, device="cuda") % 7).int()[:, None]
    w, dout = _pattern(t, 2, F32)[:, None], _pattern(t, 3)[:, None]
    row = lambda lo, hi: y.float()[pos[lo:hi, 0].long()]  # noqa: E731
    _equal(mx.moe_combine(y, pos, w), lambda lo, hi: (w[lo:hi] * row(lo, hi)).to(BF))
    log(f"moe_combine_bwd {t} x 1")
    _, dw = mx.moe_combine_bwd(dout, y, pos, w, want_dy=False)
    _equal(dw, lambda lo, hi: dout[lo:hi].float() * row(lo, hi))


def test_route_gradient():
    t = (1 << 28) + 9                   # 16 tokens a workgroup of 256
    log(f"moe_route_bwd {t} x 1")
    logits = torch.zeros((t, 1), dtype=BF, device="cuda")
    ids = torch.zeros((t, 1), dtype=torch.int32, device="cuda")
    w, d = torch.full((t, 1), 0.5, device="cuda"), _pattern(t, 4)[:, None].float()
    route = mx.Route(ids, w, None, None, None, renormalize=True)
    # w (d - w d) is exact at w = 1/2
    _equal(mx.moe_route_bwd(logits, route, d), lambda lo, hi: (d[lo:hi] / 4).to(BF))


def test_product_of_few_rows():
    n = (1 << 28) + 7                   # 16 columns a workgroup of 256
    log(f"forward 1 row 1 -> {n}")
    x, w = torch.full((1, 1), 1.5, dtype=BF, device="cuda"), _pattern(n, 5).view(1, n, 1)
    got = mx.ragged_gemm("NT", x, w, torch.tensor([1], device="cuda"))
    _equal(got[0], lambda lo, hi: w[0, lo:hi, 0] * 1.5)


def test_product_of_any_size():
    k = (1 << 31) - 1                   # 128 columns a workgroup of 256
    log(f"weight gradient 1 row 1 x {k}")
    x, dy = _pattern(k, 6).view(1, k), torch.full((1, 1), 1.5, dtype=BF, device="cuda")
    got = mx.ragged_gemm("TN", dy, x, torch.tensor([1], device="cuda"))
    _equal(got[0, 0], lambda lo, hi: x[0, lo:hi] * 1.5)
