"""Refusals of the gated products on the host: nothing here reaches a kernel."""

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


def _forward(lib, type=BF16, x=FAKE, ldx=64, w=FAKE, a=FAKE, lda=64, h=FAKE, R=8, S=8, F=64, K=64, ms=FAKE, G=2,
             index=None):
    st = lib.mxfp8_ragged_gemm_swiglu(type, x, ldx, w, a, lda, h, R, S, F, K, ms, G, index, None, 0, None)
    return st, lib.mxfp8_last_error().decode()


def _backward(lib, type=BF16, dy=FAKE, lddy=64, w=FAKE, h=FAKE, dh=FAKE, a=FAKE, R=8, N=64, F=64, ms=FAKE, G=2):
    st = lib.mxfp8_ragged_gemm_swiglu_bwd(type, dy, lddy, w, h, dh, a, R, N, F, ms, G, None, 0, None)
    return st, lib.mxfp8_last_error().decode()


def test_forward_refuses(lib):
    for t in (F32, 3, -1):
        assert _forward(lib, type=t)[0] == 2
    for kw in ({"R": -1, "S": -1}, {"F": 0}, {"F": 1 << 30, "lda": 1 << 30}, {"K": 0}, {"K": 1 << 31, "ldx": 1 << 31},
               {"G": 0}, {"G": 1025}, {"R": 1 << 31, "S": 1 << 31}, {"S": 9}, {"ms": None}, {"ldx": 63}, {"lda": 63}):
        assert _forward(lib, **kw)[0] == 1, kw


def test_backward_refuses(lib):
    for t in (F32, 3, -1):
        assert _backward(lib, type=t)[0] == 2
    for kw in ({"R": -1}, {"F": 0}, {"F": 1 << 30}, {"N": 0}, {"N": 1 << 31, "lddy": 1 << 31}, {"G": 0}, {"G": 1025},
               {"R": 1 << 31}, {"ms": None}, {"lddy": 63}):
        assert _backward(lib, **kw)[0] == 1, kw


def test_host_splits_are_refused(lib):
    splits = np.array([8], dtype=np.int64)
    at = splits.ctypes.data_as(ctypes.c_void_p)
    for call in (_forward, _backward):
        st, msg = call(lib, ms=at, G=1)
        assert st == 1 and "m_splits" in msg


def test_workspace_sizes(lib):
    size = lib.mxfp8_ragged_gemm_swiglu_workspace_bytes
    # sizes that are refused, no rows, and few rows take none
    for args in ((0, -1, 64, 64, 1), (0, 8, 0, 64, 1), (0, 8, 64, 0, 1), (1, 8, 64, 64, 0), (1, 8, 64, 64, 1025),
                 (0, 1 << 31, 64, 64, 1), (0, 8, 1 << 30, 64, 1), (0, 0, 64, 64, 1), (0, 8, 64, 64, 1)):
        assert size(*args) == 0, args
    assert size(0, 8192, 14336, 4096, 8) > 0 and size(1, 8192, 14336, 4096, 8) > 0
    assert mx.ragged_gemm_swiglu_workspace_bytes(True, 8192, 14336, 4096, 8) == size(1, 8192, 14336, 4096, 8)


def test_binding_refuses(lib):
    bf = torch.bfloat16
    x, w, w2 = torch.zeros((4, 8), dtype=bf), torch.zeros((2, 16, 8), dtype=bf), torch.zeros((2, 8, 8), dtype=bf)
    ms = torch.tensor([2, 2])
    with pytest.raises(ValueError):
        mx.ragged_gemm_swiglu(x, w, ms)                          # host splits
    with pytest.raises(ValueError):
        mx.ragged_gemm_swiglu_bwd(x, w2, torch.zeros((4, 16), dtype=bf), ms)
