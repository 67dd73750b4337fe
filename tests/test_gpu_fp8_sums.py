"""The sums of 8-bit floating-point products: fp32 in every form and for every result, few bits only where the
caller asks for fast ones."""

import ctypes

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from moe_expert_grouped_group_amd import _native
from test_gpu_ragged_fp8 import BF, F8, F32, HF, _blocks, _case, _check, _gather, _ms, _spans, _spread

pytestmark = pytest.mark.gpu


def _check_fp32_sums(q, scale, w, w_scale, splits, index, got):
    """The bound of fp32 results for every type: products of codes are exact, 128 of them are added in steps of
    at most 16, the scales' product, its product with the sum and the sum over blocks (parts of split
    tiles among them) round once each; the result is rounded once more to its type."""
    x, k = q.double() * _spread(scale, q.shape), q.shape[1]
    for e, (lo, hi) in enumerate(_spans(splits, got.shape[0])):
        if hi == lo:
            continue
        a, b = _gather(x, index)[lo:hi], w[e].double() * _spread(w_scale, w.shape)[e]
        ref, mag = a @ b.T, a.abs() @ b.abs().T
        off = mag * (12 + 2 * _blocks(k)) * 2.0 ** -23
        fin = torch.finfo(got.dtype)
        tol = off + (ref.abs() + off) * fin.eps / 2 + fin.tiny * fin.eps
        bad = ~((got[lo:hi].double() - ref).abs() <= tol)
        assert not bad.any(), (e, int(bad.sum()), float(((got[lo:hi].double() - ref).abs() / tol).max()))


def _cancelling(tokens, groups, k, n):
    """Every run of 8 along the contraction holds two large products that cancel and six small ones."""
    gen = torch.Generator("cuda").manual_seed(9)
    q = torch.rand((tokens, k), generator=gen, device="cuda") * 2 - 1
    w = torch.rand((groups, n, k), generator=gen, device="cuda") * 2 - 1
    q[:, 0::8], q[:, 1::8], w[..., 0::8], w[..., 1::8] = 256.0, 256.0, 448.0, -448.0
    scale = torch.rand((tokens, _blocks(k)), generator=gen, device="cuda") + 0.5
    w_scale = torch.rand((groups, _blocks(n), _blocks(k)), generator=gen, device="cuda") + 0.5
    return q.to(F8), scale, w.to(F8), w_scale


# (splits, K, N): few rows; tiles of 64 and of 128 rows; of 256, whole and split along the contraction; few tiles,
# split; any size
SIZES = [([1, 0, 3], 1024, 1040), ([31] * 8, 2304, 8192), ([64, 200, 120], 1296, 3000), ([300, 5, 700], 896, 5120),
         ([2000, 1900], 512, 5120), ([3000, 1, 2800], 1296, 5120), ([3320], 4112, 5120), ([300], 4112, 4096), ([96, 95], 10128, 1032), ([700, 5], 128, 256),
         ([300, 0, 65], 1031, 517)]


@pytest.mark.parametrize("out", [BF, HF, F32])
@pytest.mark.parametrize("splits,k,n", SIZES)
def test_sums_are_fp32(splits, k, n, out):
    rows = sum(splits)
    index = torch.randperm(rows, generator=torch.Generator().manual_seed(5)).int().cuda()
    case = _case(rows, splits, k, n)
    for at in (None, index):
        _check_fp32_sums(*case, splits, at, mx.ragged_gemm_fp8(*case, _ms(splits), row_index=at, out_dtype=out))


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("splits,k,n", SIZES)
def test_large_products_that_cancel(splits, k, n, out):
    case = _cancelling(sum(splits), len(splits), k, n)
    _check_fp32_sums(*case, splits, None, mx.ragged_gemm_fp8(*case, _ms(splits), out_dtype=out))


@pytest.mark.parametrize("k,n", [(640, 1024), (128, 264)])
def test_a_row_beside_few_and_many_rows(k, n):
    """A large product and its negative beside products of 1: exact in fp32 wherever the row is computed."""
    q = torch.zeros((700, k), device="cuda")
    w = torch.zeros((1, n, k), device="cuda")
    q[:, 0::8], q[:, 1::8], q[:, 2::8] = 256.0, 256.0, 1.0
    w[..., 0::8], w[..., 1::8], w[..., 2::8] = 256.0, -256.0, 1.0
    one = torch.ones((700, _blocks(k)), device="cuda"), torch.ones((1, _blocks(n), _blocks(k)), device="cuda")
    for rows in (1, 40, 300, 700):
        for out in (BF, HF, F32):
            got = mx.ragged_gemm_fp8(q[:rows].to(F8), one[0][:rows].contiguous(), w.to(F8), one[1], _ms([rows]),
                                     out_dtype=out)
            assert (got == k // 8).all(), (rows, out, got[0, :4])


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("k", [16, 128, 256, 400])
def test_many_tiles_of_few_stages(k, fast):
    """One, two and four blocks of the contraction: the copies run up to two tiles ahead of the sums."""
    splits, n = [3000, 0, 901], 5128
    rows = sum(splits)
    index = torch.randint(-1, rows + 1, (rows,), generator=torch.Generator().manual_seed(4)).int().cuda()
    case = _case(rows, splits, k, n)
    for at in (None, index):
        got = mx.ragged_gemm_fp8(*case, _ms(splits), row_index=at, fast_sums=fast)
        (_check if fast else _check_fp32_sums)(*case, splits, at, got)


@pytest.mark.parametrize("splits,k,n", SIZES)
def test_fast_sums(splits, k, n):
    """Within what 8-bit sums may lose, and the same from call to call."""
    rows = sum(splits)
    index = torch.randint(-1, rows + 1, (rows,), generator=torch.Generator().manual_seed(4)).int().cuda()
    case = _case(rows, splits, k, n)
    for out in (BF, HF):
        for at in (None, index):
            got = mx.ragged_gemm_fp8(*case, _ms(splits), row_index=at, out_dtype=out, fast_sums=True)
            _check(*case, splits, at, got)
            assert torch.equal(got, mx.ragged_gemm_fp8(*case, _ms(splits), row_index=at, out_dtype=out, fast_sums=True))
    with pytest.raises(NotImplementedError):
        mx.ragged_gemm_fp8(*case, _ms(splits), out_dtype=F32, fast_sums=True)


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("splits,k,n", [([300], 4112, 4096), ([40, 300, 0, 260], 7184, 520), ([96, 95], 10128, 1032)])
def test_without_a_workspace(splits, k, n, fast):
    """No workspace and one that is too small: nothing is split, the same result within the bounds."""
    rows = sum(splits)
    case, ms = _case(rows, splits, k, n), _ms(splits)
    lib, ptr = _native.load(), lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    fn = lib.mxfp8_ragged_gemm_fp8_fast if fast else lib.mxfp8_ragged_gemm_fp8
    assert mx.ragged_gemm_fp8_workspace_bytes(rows, rows, n, k, len(splits)) > 0
    for size in (0, 4096):
        ws = torch.full((size + 64,), 7, dtype=torch.uint8, device="cuda")
        out = torch.full((rows, n), 7.0, dtype=BF, device="cuda")
        q, scale, w, w_scale = case
        assert fn(ptr(q), k, ptr(scale), ptr(w), ptr(w_scale), ptr(out), n, 1, rows, rows, n, k, ptr(ms), len(splits),
                  None, ptr(ws) if size else None, size,
                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        torch.cuda.synchronize()
        (_check if fast else _check_fp32_sums)(*case, splits, None, out)
        assert (ws == 7).all()
