"""The gated products through the C entries without a workspace, with one that is too small and with one of the
size asked for: nothing is split, or tiles of a long contraction are; right each time."""

import ctypes

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from moe_expert_grouped_group_amd import _native
from test_gpu_ragged_swiglu import BF, HF, _check_backward, _check_forward, _ms, _normal

pytestmark = pytest.mark.gpu

# (splits, contraction, F): tiles of 64, 128 and 256 rows, fewer than CUs, and a round and a part of one; the first
# and [300, 5] have a forward product of few rows, which needs no workspace
SIZES = [([31] * 4, 4096, 1024), ([31] * 8, 2304, 2048), ([90, 0, 70], 4104, 1000), ([300], 4096, 1024), ([300, 5], 2056, 264), ([300, 301], 2056, 264),
         ([1900, 1700], 1024, 2560)]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _workspaces(need):
    """None, one of 4 KB, the size asked for; 64 bytes behind each stay as they are."""
    for size in (0, 4096, need):
        ws = torch.full((size + 64,), 7, dtype=torch.uint8, device="cuda")
        yield size, (_ptr(ws) if size else None), ws[size:]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("splits,k,f", SIZES)
def test_forward(splits, k, f, dtype):
    rows, g = sum(splits), len(splits)
    x, w, ms = _normal((rows, k), 1, dtype), _normal((g, 2 * f, k), 2, dtype, k ** -0.5), _ms(splits)
    need = mx.ragged_gemm_swiglu_workspace_bytes(False, rows, f, k, g)
    assert need > 0 or rows in (124, 305)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for size, ws, behind in _workspaces(need):
        for keep in (True, False):
            a = torch.full((rows, f), 7.0, dtype=dtype, device="cuda")
            h = torch.full((rows, 2 * f), 7.0, dtype=dtype, device="cuda") if keep else None
            assert _native.load().mxfp8_ragged_gemm_swiglu(
                1 if dtype == BF else 2, _ptr(x), k, _ptr(w), _ptr(a), f, _ptr(h), rows, rows, f, k, _ptr(ms), g, None,
                ws, size, stream) == 0
            torch.cuda.synchronize()
            _check_forward(x, w, splits, None, h, a, rows)
            assert (behind == 7).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("splits,n,f", SIZES)
def test_backward(splits, n, f, dtype):
    rows, g = sum(splits), len(splits)
    dy, w, ms = _normal((rows, n), 3, dtype), _normal((g, n, f), 4, dtype, n ** -0.5), _ms(splits)
    h = _normal((rows, 2 * f), 5, dtype)
    need = mx.ragged_gemm_swiglu_workspace_bytes(True, rows, f, n, g)
    assert need > 0
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for size, ws, behind in _workspaces(need):
        for want_a in (True, False):
            dh = torch.full((rows, 2 * f), 7.0, dtype=dtype, device="cuda")
            a = torch.full((rows, f), 7.0, dtype=dtype, device="cuda") if want_a else None
            assert _native.load().mxfp8_ragged_gemm_swiglu_bwd(
                1 if dtype == BF else 2, _ptr(dy), n, _ptr(w), _ptr(h), _ptr(dh), _ptr(a), rows, n, f, _ptr(ms), g, ws,
                size, stream) == 0
            torch.cuda.synchronize()
            _check_backward(dy, w, h, splits, dh, a)
            assert (behind == 7).all()
