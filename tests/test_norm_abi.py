"""Refusals of the norms around a block on the host: nothing here reaches a kernel."""

import math
import os

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


def _forward(lib, x=FAKE, xt=BF16, f=FAKE, t=BF16, T=4, H=64, gate=FAKE, post=FAKE, pre=FAKE, wt=F32, eps=1e-6,
             r=FAKE, y=FAKE):
    return lib.mxfp8_residual_norm(x, xt, f, t, T, H, 1.0, gate, post, pre, wt, eps, r, y, None)


def _backward(lib, dy=FAKE, dr=FAKE, r=FAKE, xt=BF16, f=FAKE, t=BF16, T=4, H=64, gate=FAKE, post=FAKE, pre=FAKE,
              wt=F32, eps=1e-6, dx=FAKE, df=FAKE, dgate=FAKE, dpost=FAKE, dpre=FAKE, ws=FAKE, size=1 << 30):
    return lib.mxfp8_residual_norm_bwd(dy, dr, r, xt, f, t, T, H, 1.0, gate, post, pre, wt, eps, dx, df, dgate,
                                       dpost, dpre, ws, size, None)


BOTH = ({"T": -1}, {"T": 1 << 31}, {"H": 0}, {"H": 16385}, {"eps": -1e-6}, {"eps": math.nan}, {"eps": math.inf},
        {"f": FAKE + 1}, {"gate": FAKE + 2}, {"post": FAKE + 2}, {"pre": FAKE + 2}, {"wt": BF16, "pre": FAKE + 1})


def test_forward_refuses(lib):
    for kw in ({"t": F32}, {"t": 3}, {"xt": F16}, {"xt": BF16, "t": F16}, {"wt": F16}, {"wt": -1}):
        assert _forward(lib, **kw) == 2, kw
    for kw in BOTH + ({"x": None}, {"f": None}, {"f": None, "gate": None, "post": None}, {"r": None}, {"y": None},
                      {"pre": None}, {"f": None, "gate": None, "post": None, "r": None, "pre": None, "y": None},
                      {"xt": F32, "x": FAKE + 2}, {"xt": F32, "r": FAKE + 2}, {"y": FAKE + 1}):
        assert _forward(lib, **kw) == 1, kw
    assert _forward(lib, T=0, x=None, f=None, r=None, y=None) == 0


def test_backward_refuses(lib):
    for kw in ({"t": F32}, {"xt": F16}, {"wt": F16}):
        assert _backward(lib, **kw) == 2, kw
    none = {"dx": None, "df": None, "dgate": None, "dpost": None, "dpre": None}
    for kw in BOTH + (none, {"post": None}, {"gate": None}, {"pre": None}, {"ws": None}, {"size": 16}, {"ws": FAKE + 2},
                      {"dy": None, "dr": None}, {"dy": None}, {"r": None}, {"f": None, "gate": None, "post": None},
                      {"pre": None, "dpre": None}, {"xt": F32, "dx": FAKE + 2}, {"df": FAKE + 1}, {"dgate": FAKE + 2}):
        assert _backward(lib, **kw) == 1, kw


def test_workspace_sizes(lib):
    size = lib.mxfp8_residual_norm_bwd_workspace_bytes
    for args in ((-1, 64), (4, 0), (4, 16385), (1 << 31, 64), (0, 64)):
        assert size(*args) == 0, args
    assert size(1, 64) >= 2 * 64 * 4 and size(1 << 30, 4096) < 1 << 28
    assert mx.residual_norm_bwd_workspace_bytes(100, 4096) == size(100, 4096)


def test_binding_refuses(lib):
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    w = torch.ones(8)
    for call in (lambda: mx.residual_norm(x, x, pre_weight=w),             # host tensors
                 lambda: mx.residual_norm(x[0], pre_weight=w),
                 lambda: mx.residual_norm(x, gate=torch.ones(4), pre_weight=w),   # gate without f
                 lambda: mx.residual_norm(x, post_weight=w, pre_weight=w),
                 lambda: mx.residual_norm_bwd(x, x, x, gate=torch.ones(4), pre_weight=w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mx.residual_norm(x, x.float(), pre_weight=w),
                 lambda: mx.residual_norm(x, x.half(), pre_weight=w),
                 lambda: mx.residual_norm(x.half(), x, pre_weight=w),
                 lambda: mx.residual_norm(x, pre_weight=w, out_dtype=torch.float32)):
        with pytest.raises(NotImplementedError):
            call()
