"""Row indexes outside the source stand for a row of zeros in every form of the
ragged products: the results are those of a source that has such a row, so zero
times a weight that is infinite or NaN is NaN, whichever form the sizes choose."""

import math

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from gpu_util import log

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

# K, N, splits: few rows (16, 32 and 64 of them a workgroup, short and long runs, many
# workgroups and few), any alignment, large tiles of 64, 128 and 256 rows
SIZES = [(40, 24, [3, 2]), (2056, 16400, [5, 1]), (1031, 517, [1, 4]), (136, 264, [30, 0, 31]),
         (64, 256, [60, 200]), (37, 50, [300, 301]), (264, 72, [300, 301]),
         (6152, 4104, [20, 0, 41, 1, 64, 33]), (6208, 4136, [63, 65, 0, 130, 100, 1])]
SIZES_INT8 = SIZES[:7] + [(12304, 4104, [20, 0, 41, 1, 64, 33]), (12416, 4136, [63, 65, 0, 130, 100, 1])]


def _normal(shape, seed, dtype):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _index(rows, tokens):
    """Every third row has no token."""
    index = torch.arange(rows, device="cuda") % tokens
    off = torch.tensor([-1, tokens, -(1 << 31), (1 << 31) - 1], device="cuda")
    gone = torch.arange(rows, device="cuda") % 3 == 0
    return torch.where(gone, off[torch.arange(rows, device="cuda") % 4], index).int(), gone


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("k,n,splits", SIZES)
def test_forward(k, n, splits, out):
    log(f"forward {k} x {n} {splits} {out}")
    rows, g = sum(splits), len(splits)
    x, w = _normal((7, k), 1, BF), _normal((g, n, k), 2, BF)
    w[:, 3, 5], w[:, n - 1, k - 1], w[:, n // 2, 0] = math.inf, math.nan, -math.inf
    index, gone = _index(rows, 7)
    got = mx.ragged_gemm("NT", x, w, torch.tensor(splits, device="cuda"), row_index=index, out_dtype=out)
    expect = torch.zeros(n, dtype=torch.bool, device="cuda")
    expect[[3, n - 1, n // 2]] = True
    assert torch.equal(torch.isnan(got[gone]), expect.expand(int(gone.sum()), n))
    assert (got[gone][:, ~expect] == 0).all()
    # the others' rows are finite where the weights are
    assert torch.isfinite(got[~gone][:, ~expect]).all() and not torch.isfinite(got[~gone][:, expect]).any()


@pytest.mark.parametrize("k,n,splits", SIZES_INT8)
def test_int8(k, n, splits):
    """A channel's scale that is NaN or infinite (as quantize_int8 makes of one that
    holds an infinity)."""
    log(f"int8 {k} x {n} {splits}")
    rows, g = sum(splits), len(splits)
    gen = torch.Generator("cuda").manual_seed(1)
    q = torch.randint(-127, 128, (7, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (g, n, k), generator=gen, device="cuda", dtype=torch.int8)
    sc, ws = torch.rand(7, generator=gen, device="cuda"), torch.rand((g, n), generator=gen, device="cuda")
    ws[:, 3], ws[:, n - 1] = math.nan, math.inf
    index, gone = _index(rows, 7)
    got = mx.ragged_gemm_int8(q, sc, w, ws, torch.tensor(splits, device="cuda"), row_index=index)
    expect = torch.zeros(n, dtype=torch.bool, device="cuda")
    expect[[3, n - 1]] = True
    assert torch.equal(torch.isnan(got[gone]), expect.expand(int(gone.sum()), n))
    assert (got[gone][:, ~expect] == 0).all()
    assert torch.isfinite(got[~gone][:, ~expect]).all()


@pytest.mark.parametrize("k,n,splits", [(37, 50, [300, 301]), (264, 72, [300, 301]), (40, 24, [3, 2])])
def test_weight_gradient(k, n, splits):
    log(f"weight gradient {k} x {n} {splits}")
    rows, g = sum(splits), len(splits)
    x, dy = _normal((7, k), 1, BF), _normal((rows, n), 2, BF)
    index, gone = _index(rows, 7)
    clean = mx.ragged_gemm("TN", dy, x, torch.tensor(splits, device="cuda"), row_index=index)
    assert torch.isfinite(clean).all()
    dy[0, 4] = math.inf                 # row 0 of expert 0 has no token
    got = mx.ragged_gemm("TN", dy, x, torch.tensor(splits, device="cuda"), row_index=index)
    assert torch.isnan(got[0, 4]).all()
    got[0, 4] = clean[0, 4]
    assert torch.equal(got, clean)
