"""Large tiles that follow one another in a workgroup.  With more tiles than the 256
workgroups and contractions of some stages (of 128 bytes), the last stages of a tile carry
the first copies of the next one, with its row indexes and scales; the tiles past
the last full round are split along the contraction.  All sizes here have both.

Small whole numbers: sums are exact in fp32 and the output's rounding is the only one, so
results are equal to float64 ones rounded once."""

import math

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from gpu_util import log

pytestmark = pytest.mark.gpu

BF, HF, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
PAST = 5     # rows past the last expert's


def _whole(shape, seed, dtype, most=4):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").to(dtype)


def _spans(splits):
    ends = [sum(splits[:i + 1]) for i in range(len(splits))]
    return list(zip([0] + ends[:-1], ends))


def _index(rows, tokens, seed):
    """Any token any number of times; a few rows without one, none past the experts'."""
    gen = torch.Generator("cuda").manual_seed(seed)
    index = torch.randint(0, tokens, (rows,), generator=gen, device="cuda").int()
    index[::37], index[5::61] = -1, tokens
    index[rows - PAST:] = -1
    return index


def _rows(x, index):
    """Rows in float64; an index outside gives zeros."""
    at = index.long()
    ok = (at >= 0) & (at < len(x))
    return torch.where(ok[:, None], x[at.clamp(0, len(x) - 1)].double(), 0.0)


# splits, N, tiles: 264 of 256 rows (the last 8 in 4 parts), 273 of 64 and of 128 rows (17 in 2)
TALL = ([700, 0, 1, 1281, 512], 5608)
FORWARD = {"256 rows": (*TALL, 1544), "64 rows": ([60, 0, 100, 1, 7, 64, 0, 8], 9736, 1288),
           "128 rows": ([129, 0, 200, 64, 1, 26], 9736, 1288)}


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", FORWARD)
def test_forward(name, gather, dtype):
    splits, n, k = FORWARD[name]
    log(f"forward {name} gather={gather} {dtype}")
    rows, g = sum(splits) + PAST, len(splits)
    x, w = _whole((rows, k), 1, dtype), _whole((g, n, k), 2, dtype)
    index = _index(rows, rows, 3) if gather else None
    if not gather:
        x[rows - PAST:] = math.nan
    xr = _rows(x, index) if gather else x.double()
    for out in (dtype, F32):
        y = torch.full((rows, n), 7.0, dtype=out, device="cuda")
        mx.ragged_gemm("NT", x, w, torch.tensor(splits, device="cuda"), row_index=index, out=y, out_dtype=out)
        for i, (lo, hi) in enumerate(_spans(splits)):
            assert torch.equal(y[lo:hi], (xr[lo:hi] @ w[i].double().T).to(out)), i
        assert (y[rows - PAST:] == 7.0).all()


@pytest.mark.parametrize("out", [F32, BF, HF])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", FORWARD)
def test_int8(name, gather, out):
    """The integer sum, rounded to fp32, times two scales in their order."""
    splits, n, k = FORWARD[name]
    k = 2 * k
    log(f"int8 {name} gather={gather} {out}")
    rows, g = sum(splits) + PAST, len(splits)
    gen = torch.Generator("cuda").manual_seed(4)
    q, w = _whole((rows, k), 1, I8, 127), _whole((g, n, k), 2, I8, 127)
    sc, ws = torch.rand(rows, generator=gen, device="cuda") * 1e-2, torch.rand((g, n), generator=gen, device="cuda")
    index = _index(rows, rows, 3) if gather else None
    qr = _rows(q, index) if gather else q.double()
    sr = _rows(sc[:, None], index)[:, 0].float() if gather else sc
    y = torch.full((rows, n), 7.0, dtype=out, device="cuda")
    mx.ragged_gemm_int8(q, sc, w, ws, torch.tensor(splits, device="cuda"), row_index=index, out=y, out_dtype=out)
    for i, (lo, hi) in enumerate(_spans(splits)):
        ref = (qr[lo:hi] @ w[i].double().T).float() * sr[lo:hi, None] * ws[i]
        assert torch.equal(y[lo:hi], ref.to(out)), i
    assert (y[rows - PAST:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_input_gradient(dtype):
    splits, k = TALL
    n = 1544
    log(f"input gradient {dtype}")
    rows, g = sum(splits) + PAST, len(splits)
    dy, w = _whole((rows, n), 1, dtype), _whole((g, n, k), 2, dtype)
    dy[rows - PAST:] = math.nan
    for out in (dtype, F32):
        dx = torch.full((rows, k), 7.0, dtype=out, device="cuda")
        mx.ragged_gemm("NN", dy, w, torch.tensor(splits, device="cuda"), out=dx, out_dtype=out)
        for i, (lo, hi) in enumerate(_spans(splits)):
            assert torch.equal(dx[lo:hi], (dy[lo:hi].double() @ w[i].double()).to(out)), i
        assert (dx[rows - PAST:] == 7.0).all()


# splits, N, K: 264 tiles, the last 8, of the last expert, in 2 parts; 9 tiles in 7 parts; 5 in 2,
# of experts that have no stage, one (so none for the second part), three, and a last one of one row
WGRAD = [([0, 20, 700, 1280], 1496, 2696), ([5003], 520, 520), ([3, 0, 2500, 65, 129], 200, 248)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("splits,n,k", WGRAD)
def test_weight_gradient(splits, n, k, gather, dtype):
    log(f"weight gradient {splits} {n} x {k} gather={gather} {dtype}")
    rows, g = sum(splits) + PAST, len(splits)
    x, dy = _whole((rows if not gather else 901, k), 1, dtype), _whole((rows, n), 2, dtype)
    dy[rows - PAST:] = math.nan
    index = _index(rows, len(x), 3) if gather else None
    if not gather:
        x[rows - PAST:] = math.nan
    xr = _rows(x, index) if gather else x.double()
    for out in (dtype, F32):
        got = mx.ragged_gemm("TN", dy, x, torch.tensor(splits, device="cuda"), row_index=index, out_dtype=out)
        for i, (lo, hi) in enumerate(_spans(splits)):
            assert torch.equal(got[i], (dy[lo:hi].double().T @ xr[lo:hi]).to(out)), i
