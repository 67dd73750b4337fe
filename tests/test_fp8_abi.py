"""Refusals of the 8-bit floating point calls on the host: nothing here reaches a kernel."""

import ctypes
import os

import numpy as np
import pytest
import torch

import moe_expert_grouped_group_amd as mx
from moe_expert_grouped_group_amd import _native

FAKE = 0x1000  # never dereferenced: every call below fails validation first
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.lib_path()):
        from moe_expert_grouped_group_amd import build
        build.build()
    return _native.load()


def test_quantize_refuses(lib):
    f = lib.mxfp8_quantize_fp8
    assert f(FAKE, F32, 4, 8, 8, FAKE, FAKE, None) == 2
    for args in ((FAKE, BF16, -1, 8, 8, FAKE, FAKE), (FAKE, BF16, 4, 0, 8, FAKE, FAKE),
                 (FAKE, BF16, 4, 8, 7, FAKE, FAKE), (None, BF16, 4, 8, 8, FAKE, FAKE),
                 (FAKE, BF16, 4, 8, 8, None, FAKE), (FAKE, BF16, 4, 8, 8, FAKE, None),
                 (FAKE, BF16, 1 << 31, 8, 8, FAKE, FAKE), (FAKE, BF16, 1, 1 << 31, 1 << 31, FAKE, FAKE),
                 (FAKE + 1, BF16, 4, 8, 8, FAKE, FAKE), (FAKE, BF16, 4, 8, 8, FAKE, FAKE + 2)):
        assert f(*args, None) == 1, args
    assert f(None, F16, 0, 8, 8, None, None, None) == 0


def test_quantize_weight_refuses(lib):
    f = lib.mxfp8_quantize_fp8_weight
    assert f(FAKE, F32, 4, 8, 8, FAKE, FAKE, None) == 2
    for args in ((FAKE, BF16, -1, 8, 8, FAKE, FAKE), (FAKE, BF16, 4, 0, 8, FAKE, FAKE),
                 (FAKE, BF16, 4, 8, 0, FAKE, FAKE), (None, BF16, 4, 8, 8, FAKE, FAKE),
                 (FAKE, BF16, 4, 8, 8, None, FAKE), (FAKE, BF16, 4, 8, 8, FAKE, None),
                 (FAKE, BF16, 1 << 31, 8, 8, FAKE, FAKE), (FAKE, BF16, 1, (1 << 31) - 1, (1 << 31) - 1, FAKE, FAKE),
                 (FAKE, BF16, (1 << 31) - 1, 1 << 20, 1 << 20, FAKE, FAKE),
                 (FAKE + 1, BF16, 4, 8, 8, FAKE, FAKE), (FAKE, BF16, 4, 8, 8, FAKE, FAKE + 2)):
        assert f(*args, None) == 1, args
    assert f(None, F16, 0, 8, 8, None, None, None) == 0


def _gemm(lib, q=FAKE, ldq=64, sc=FAKE, w=FAKE, ws=FAKE, c=FAKE, ldc=64, ct=BF16, R=8, S=8, N=64, K=64, ms=FAKE, G=2,
          index=None):
    st = lib.mxfp8_ragged_gemm_fp8(q, ldq, sc, w, ws, c, ldc, ct, R, S, N, K, ms, G, index, None, 0, None)
    return st, lib.mxfp8_last_error().decode()


def test_gemm_refuses(lib):
    for t in (3, -1):
        assert _gemm(lib, ct=t)[0] == 2
    for kw in ({"R": -1, "S": -1}, {"N": 0}, {"K": 0}, {"G": 0}, {"G": 1025}, {"R": 1 << 31, "S": 1 << 31},
               {"N": 1 << 31, "ldc": 1 << 31}, {"K": 1 << 31, "ldq": 1 << 31}, {"S": 9}, {"ms": None}, {"ldq": 63},
               {"ldc": 63}):
        assert _gemm(lib, **kw)[0] == 1, kw
    splits = np.array([8], dtype=np.int64)
    st, msg = _gemm(lib, ms=splits.ctypes.data_as(ctypes.c_void_p), G=1)
    assert st == 1 and "m_splits" in msg


def test_workspace_sizes(lib):
    size = lib.mxfp8_ragged_gemm_fp8_workspace_bytes
    for args in ((-1, 8, 64, 64, 1), (8, -1, 64, 64, 1), (8, 8, 0, 64, 1), (8, 8, 64, 0, 1), (8, 8, 64, 64, 0),
                 (8, 8, 64, 64, 1025), (1 << 31, 8, 64, 64, 1), (0, 0, 64, 64, 1), (8, 8, 64, 64, 1)):
        assert size(*args) == 0, args


def test_binding_refuses(lib):
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(NotImplementedError):
        mx.quantize_fp8(x.float())
    with pytest.raises(ValueError):
        mx.quantize_fp8(x)                                       # host tensor
    with pytest.raises(ValueError):
        mx.quantize_fp8(x[0])
    with pytest.raises(ValueError):
        mx.quantize_fp8_weight(x)                                # not [G, N, K]
    with pytest.raises(ValueError):
        mx.ragged_gemm_fp8(x.to(torch.float8_e4m3fn), torch.zeros((4, 1)), x[None].to(torch.float8_e4m3fn),
                           torch.zeros((1, 1, 1)), torch.tensor([4]))   # host splits


def test_fast_gemm_refuses(lib):
    """As the other one, and fp32 results."""
    def call(ct=BF16, R=8, q=FAKE, ldq=64, S=8):
        return lib.mxfp8_ragged_gemm_fp8_fast(q, ldq, FAKE, FAKE, FAKE, FAKE, 64, ct, R, S, 64, 64, FAKE, 2, None, None, 0,
                                              None)
    for ct in (F32, 3, -1):
        assert call(ct=ct) == 2
    assert "mxfp8_ragged_gemm_fp8_fast" in lib.mxfp8_last_error().decode()
    for kw in ({"R": -1}, {"q": None}, {"ldq": 63}, {"S": 9}):
        assert call(**kw) == 1, kw
