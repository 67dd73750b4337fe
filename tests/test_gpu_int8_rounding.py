"""The roundings of the 8-bit product, one by one: the exact sum to fp32, each of the two
scales' products to fp32, then the output's type.  Bit-equal in every form and type."""

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from gpu_util import log

pytestmark = pytest.mark.gpu

# K, N, splits: few rows (16, 32, 64 a workgroup; short and long runs), any size, rows laid
# out anew, large tiles of 64, 128 and 256 rows
SIZES = [(1000, 1031, [7, 0, 5]), (8208, 16400, [3, 2]), (144, 4104, [30, 31]), (400, 2056, [60, 200]),
         (259, 1031, [300, 301]), (2111, 4011, [1200, 0, 1, 900]), (12304, 4104, [20, 0, 41, 1, 64, 33]),
         (12416, 4136, [63, 65, 0, 130, 100, 1]), (1040, 2056, [500, 700])]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("k,n,splits", SIZES)
def test_each_step_is_rounded(k, n, splits, out):
    log(f"int8 {k} x {n} {splits} {out}")
    rows, g = sum(splits), len(splits)
    gen = torch.Generator("cuda").manual_seed(1)
    q = torch.randint(-127, 128, (rows, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (g, n, k), generator=gen, device="cuda", dtype=torch.int8)
    sc = torch.rand(rows, generator=gen, device="cuda") * 1e-3
    ws = torch.rand((g, n), generator=gen, device="cuda")
    got = mx.ragged_gemm_int8(q, sc, w, ws, torch.tensor(splits, device="cuda"), out_dtype=out)
    lo = 0
    for i, m in enumerate(splits):
        ref = (q[lo:lo + m].double() @ w[i].double().T).float() * sc[lo:lo + m, None]
        ref = (ref * ws[i]).to(out)
        assert torch.equal(got[lo:lo + m], ref), i
        lo += m
