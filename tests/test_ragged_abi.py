"""Refusals of the ragged products and of the routing, on the host: nothing
here reaches a kernel."""

import ctypes
import os

import numpy as np
import pytest
import torch

import moe_expert_grouped_group_amd as mx
from moe_expert_grouped_group_amd import _native

FAKE = 0x1000  # never dereferenced: every call below fails validation first
NT, NN, TN = 0, 1, 2
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.lib_path()):
        from moe_expert_grouped_group_amd import build
        build.build()
    return _native.load()


def _gemm(lib, layout=NT, type=BF16, a=FAKE, lda=64, b=FAKE, ldb=64, c=FAKE, ldc=64, c_type=BF16, R=8, S=8,
          N=64, K=64, ms=FAKE, G=2, index=None):
    st = lib.mxfp8_ragged_gemm(layout, type, a, lda, b, ldb, c, ldc, c_type, R, S, N, K, ms, G, index, None, 0, None)
    return st, lib.mxfp8_last_error().decode()


def test_gemm_refuses(lib):
    assert _gemm(lib, layout=3)[0] == 1
    for t in (F32, 3, -1):
        assert _gemm(lib, type=t)[0] == 2
    assert _gemm(lib, type=BF16, c_type=F16)[0] == 2
    assert _gemm(lib, type=F16, c_type=BF16)[0] == 2
    for kw in ({"R": -1, "S": -1}, {"N": 0}, {"K": 0}, {"G": 0}, {"G": 1025}, {"R": 1 << 31, "S": 1 << 31},
               {"N": 1 << 31}, {"K": 1 << 31, "lda": 1 << 31}, {"S": 9}, {"ms": None},
               {"layout": NN, "index": FAKE}):
        assert _gemm(lib, **kw)[0] == 1, kw
    # tiles past the grid's limit
    assert _gemm(lib, layout=TN, N=(1 << 31) - 1, lda=1 << 31, K=1 << 20, ldb=1 << 20)[0] == 1


def test_gemm_refuses_host_splits(lib):
    splits = np.array([8], dtype=np.int64)
    st, msg = _gemm(lib, ms=splits.ctypes.data_as(ctypes.c_void_p), G=1)
    assert st == 1 and "m_splits" in msg


def test_quantize_refuses(lib):
    q = lib.mxfp8_quantize_int8
    assert q(FAKE, F32, 4, 8, 8, FAKE, FAKE, None) == 2
    for args in ((FAKE, BF16, -1, 8, 8, FAKE, FAKE), (FAKE, BF16, 4, 0, 8, FAKE, FAKE),
                 (FAKE, BF16, 4, 8, 7, FAKE, FAKE), (None, BF16, 4, 8, 8, FAKE, FAKE),
                 (FAKE, BF16, 4, 8, 8, None, FAKE), (FAKE, BF16, 4, 8, 8, FAKE, None),
                 (FAKE + 1, BF16, 4, 8, 8, FAKE, FAKE), (FAKE, BF16, 4, 8, 8, FAKE, FAKE + 2)):
        assert q(*args, None) == 1, args
    assert q(None, F16, 0, 8, 8, None, None, None) == 0


def test_int8_gemm_refuses(lib):
    def call(q=FAKE, ldq=64, sc=FAKE, w=FAKE, ws=FAKE, c=FAKE, ldc=64, ct=BF16, R=8, S=8, N=64, K=64, ms=FAKE,
             G=2, index=None):
        return lib.mxfp8_ragged_gemm_int8(q, ldq, sc, w, ws, c, ldc, ct, R, S, N, K, ms, G, index, None, 0, None)
    assert call(ct=3) == 2
    for kw in ({"N": 0}, {"K": 0}, {"G": 0}, {"G": 2000}, {"S": 9}, {"ms": None}, {"R": -1, "S": -1}):
        assert call(**kw) == 1, kw


def test_route_refuses(lib):
    def call(z=FAKE, ty=F32, T=300, E=8, k=2, mask=None, ids=FAKE, w=FAKE, ms=FAKE, tok=FAKE, pos=FAKE, ws=FAKE,
             n=1 << 20):
        return lib.mxfp8_moe_route(z, ty, T, E, k, 1, mask, ids, w, ms, tok, pos, ws, n, None)
    assert call(ty=3) == 2
    for kw in ({"E": 0}, {"E": 1025}, {"k": 0}, {"k": 9}, {"k": 17, "E": 64}, {"T": -1}, {"T": 1 << 31}, {"ms": None},
               {"z": None}, {"ids": None}, {"w": None}, {"tok": None}, {"pos": None}, {"ws": None}, {"n": 1},
               {"z": FAKE + 2}, {"ms": FAKE + 4}):
        assert call(**kw) == 1, kw
    assert lib.mxfp8_moe_route_workspace_bytes(0, 8) == 0
    assert lib.mxfp8_moe_route_workspace_bytes(100000, 8) > 0
    b = lib.mxfp8_moe_route_bwd
    assert b(FAKE, 3, 4, 8, 2, 1, FAKE, FAKE, FAKE, FAKE, None) == 2
    assert b(FAKE, F32, 4, 8, 9, 1, FAKE, FAKE, FAKE, FAKE, None) == 1
    for i in (0, 6, 7, 8, 9):
        args = [FAKE, F32, 4, 8, 2, 1, FAKE, FAKE, FAKE, FAKE]
        args[i] = None
        assert b(*args, None) == 1, i
    assert b(None, F32, 0, 8, 2, 1, None, None, None, None, None) == 0


def test_join_refuses(lib):
    f, b = lib.mxfp8_moe_combine, lib.mxfp8_moe_combine_bwd
    assert f(FAKE, F32, 4, 8, 8, 2, FAKE, None, FAKE, None) == 2
    assert b(FAKE, FAKE, F32, 4, 8, 8, 2, FAKE, None, FAKE, FAKE, None) == 2
    for T, R, H, k in ((-1, 8, 8, 2), (4, -1, 8, 2), (4, 8, 0, 2), (4, 8, 8, 0), (4, 8, 8, 17)):
        assert f(FAKE, BF16, T, R, H, k, FAKE, None, FAKE, None) == 1
        assert b(FAKE, FAKE, BF16, T, R, H, k, FAKE, None, FAKE, FAKE, None) == 1
    assert f(None, BF16, 4, 8, 8, 2, FAKE, None, FAKE, None) == 1
    assert f(FAKE, BF16, 4, 8, 8, 2, None, None, FAKE, None) == 1
    assert f(FAKE, BF16, 4, 8, 8, 2, FAKE, None, None, None) == 1
    assert b(FAKE, FAKE, BF16, 4, 8, 8, 2, FAKE, None, None, None, None) == 1
    assert b(None, FAKE, BF16, 4, 8, 8, 2, FAKE, None, FAKE, FAKE, None) == 1
    assert b(FAKE, None, BF16, 4, 8, 8, 2, FAKE, None, FAKE, FAKE, None) == 1
    assert f(None, BF16, 0, 0, 8, 2, None, None, None, None) == 0


def test_binding_refuses(lib):
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    w = torch.zeros((2, 8, 8), dtype=torch.bfloat16)
    ms = torch.tensor([2, 2])
    with pytest.raises(ValueError):
        mx.ragged_gemm("NT", x, w, ms)                       # host splits
    with pytest.raises(NotImplementedError):
        mx.quantize_int8(x.float())
    with pytest.raises(ValueError):
        mx.quantize_int8(x)                                  # host tensor
    with pytest.raises(ValueError):
        mx.quantize_int8(x[0])
    with pytest.raises(NotImplementedError):
        mx.moe_route(torch.zeros((4, 8), dtype=torch.float64), 2)
    with pytest.raises(ValueError):
        mx.moe_route(torch.zeros((4, 8)), 2)
    with pytest.raises(NotImplementedError):
        mx.moe_combine(x.float(), torch.zeros((2, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        mx.moe_combine(x, torch.zeros((2, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        mx.moe_combine_bwd(x, x, torch.zeros((2, 2), dtype=torch.int32))


def test_workspace_queries_of_refused_sizes(lib):
    """0, whatever the sizes: callers ask before the entry itself refuses."""
    route, gemm = lib.mxfp8_moe_route_workspace_bytes, lib.mxfp8_ragged_gemm_workspace_bytes
    for t, e in ((300, 10000), (300, 1025), (300, 0), (300, -1), (-1, 8), (1 << 31, 8), ((1 << 63) - 1, 1024),
                 (300, (1 << 31) - 1)):
        assert route(t, e) == 0, (t, e)
    assert route((1 << 31) - 1, 1024) > 0
    assert gemm(NN, 2, 300, 300, 64, 64, 1024) > 0
    for args in ((NN, 2, 300, 300, 64, 64, 1025), (NN, 2, 300, 300, 64, 64, 0), (NN, 2, -1, 300, 64, 64, 2),
                 (NN, 2, 300, 300, 0, 64, 2), (3, 2, 300, 300, 64, 64, 2), (NN, 4, 300, 300, 64, 64, 2)):
        assert gemm(*args) == 0, args


def test_route_of_too_many_experts_raises(lib, monkeypatch):
    """The whole call on logits [300, 10000]: a ValueError from the entry."""
    from moe_expert_grouped_group_amd import binding

    class DeviceTensor(torch.Tensor):
        is_cuda = True

    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: real(*a, **kw).as_subclass(DeviceTensor))
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    with pytest.raises(ValueError, match="E = 10000"):
        mx.moe_route(torch.zeros((300, 10000)).as_subclass(DeviceTensor), 2)


@pytest.mark.parametrize("g,n,k,size,rows,few", [
    (1, 4096, 4096, 2, 16, True), (1, 4096, 4096, 2, 64, True), (1, 4096, 4096, 2, 192, False),
    (8, 2048, 2048, 2, 64, True), (8, 2048, 2048, 2, 96, False),
    (4, 4096, 4096, 2, 20, True), (4, 4096, 4096, 2, 32, False),
    (4, 7168, 4096, 2, 12, True), (4, 7168, 4096, 2, 24, False),
    (64, 2048, 1024, 2, 8, True), (64, 2048, 1024, 2, 16, False),
    (8, 14336, 4096, 2, 4, True), (8, 14336, 4096, 2, 8, False),
    (8, 14336, 4096, 1, 8, True), (8, 14336, 4096, 1, 16, False)])
def test_form_that_measured_faster(lib, g, n, k, size, rows, few):
    """The rule between the few-rows form, which uses no workspace, and the large tiles,
    at sizes where both were timed and differ."""
    need = lib.mxfp8_ragged_gemm_workspace_bytes(NT, size, g * rows, g * rows, n, k, g)
    assert (need == 0) == few


@pytest.mark.parametrize("layout,size,g,rows,n,k,anew", [
    (NT, 2, 8, 16384, 14331, 4091, True), (NT, 2, 5, 1777, 517, 1031, False), (NT, 2, 3, 3000, 2011, 1031, False),
    (NT, 2, 4, 4000, 1003, 4011, True), (NT, 2, 1, 600, 4099, 1003, False), (NT, 2, 8, 9000, 777, 2051, False),
    (NT, 2, 64, 20000, 1021, 515, False), (NT, 1, 8, 16384, 14331, 4091, True), (NT, 1, 4, 4000, 1003, 4011, False),
    (NN, 2, 8, 16384, 14331, 4091, True), (NN, 2, 5, 1777, 517, 1031, False), (NN, 2, 3, 3000, 2011, 1031, True),
    (NN, 2, 1, 600, 4099, 1003, True), (NN, 2, 8, 9000, 777, 2051, True), (NN, 2, 2, 9000, 1501, 517, True),
    (NN, 2, 64, 20000, 1021, 515, True), (TN, 2, 8, 16384, 14331, 4091, True), (TN, 2, 5, 1777, 517, 1031, False),
    (TN, 2, 3, 3000, 2011, 1031, True), (TN, 2, 1, 600, 4099, 1003, True), (TN, 2, 64, 20000, 1021, 515, True)])
def test_layout_anew_that_measured_faster(lib, layout, size, g, rows, n, k, anew):
    """The rule that lays odd operands out anew, for which it takes more workspace than
    aligned ones, at sizes where both ways were timed."""
    ask = lib.mxfp8_ragged_gemm_workspace_bytes
    odd, even = ask(layout, size, rows, rows, n, k, g), ask(layout, size, rows, rows, n // 16 * 16, k // 16 * 16, g)
    assert (odd > even) == anew
