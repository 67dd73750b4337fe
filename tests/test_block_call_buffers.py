"""Which pool the buffers of the gated, 8-bit floating-point and norm calls come from, and
which workspaces they refuse, on the host: nothing here reaches the library or a GPU."""

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from moe_expert_grouped_group_amd import binding
from test_call_buffers import BF, F32, U8, Stream, T, _ms, pools  # noqa: F401

F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def anywhere(monkeypatch):
    """Host tensors pass for ones of the current device; no size is kept beyond a test."""
    monkeypatch.setattr(binding, "_on_current", lambda *args: None)
    sizes = (binding.ragged_gemm_swiglu_workspace_bytes, binding.ragged_gemm_fp8_workspace_bytes,
             binding.residual_norm_bwd_workspace_bytes)
    for size in sizes:
        size.cache_clear()
    yield
    for size in sizes:
        size.cache_clear()


def _norm_bwd(**kw):
    return mx.residual_norm_bwd(T(6, 8), T(6, 8), T(6, 8), T(6, 8), gate=T(6, dtype=F32), post_weight=T(8, dtype=F32),
                                pre_weight=T(8, dtype=F32), **kw)


def _fp8(**kw):
    return mx.ragged_gemm_fp8(T(8, 16, dtype=F8), T(8, 1, dtype=F32), T(2, 24, 16, dtype=F8), T(2, 1, 1, dtype=F32),
                              _ms(), **kw)


# call, buffers that it returns, workspaces that it makes
CALLS = {
    "ragged_gemm_swiglu": (lambda s: mx.ragged_gemm_swiglu(T(8, 16), T(2, 48, 16), _ms(), stream=s), 2, 1),
    "ragged_gemm_swiglu alone": (lambda s: mx.ragged_gemm_swiglu(
        T(8, 16), T(2, 48, 16), _ms(), want_h=False, stream=s), 1, 1),
    "ragged_gemm_swiglu_bwd": (lambda s: mx.ragged_gemm_swiglu_bwd(
        T(8, 24), T(2, 24, 16), T(8, 32), _ms(), stream=s), 2, 1),
    "quantize_fp8": (lambda s: mx.quantize_fp8(T(8, 16), stream=s), 2, 0),
    "quantize_fp8_weight": (lambda s: mx.quantize_fp8_weight(T(2, 8, 16), stream=s), 2, 0),
    "ragged_gemm_fp8": (lambda s: _fp8(stream=s), 1, 1),
    "residual_norm": (lambda s: mx.residual_norm(T(6, 8), T(6, 8), pre_weight=T(8, dtype=F32), stream=s), 2, 0),
    "residual_norm_bwd": (lambda s: _norm_bwd(stream=s), 5, 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_given_stream(pools, name):  # noqa: F811
    call, returned, scratch = CALLS[name]
    call(Stream("given"))
    assert len(pools) == returned + scratch
    assert {pool for pool, _ in pools} == {"given"}
    assert sum(told == {"current"} for _, told in pools) >= returned


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_current_stream(pools, name):  # noqa: F811
    call, returned, scratch = CALLS[name]
    call(None)
    assert len(pools) == returned + scratch
    assert {pool for pool, _ in pools} == {"current"}


TAKES = {
    "ragged_gemm_swiglu": lambda w: mx.ragged_gemm_swiglu(T(8, 16), T(2, 48, 16), _ms(), workspace=w),
    "ragged_gemm_swiglu_bwd": lambda w: mx.ragged_gemm_swiglu_bwd(
        T(8, 24), T(2, 24, 16), T(8, 32), _ms(), workspace=w),
    "ragged_gemm_fp8": lambda w: _fp8(workspace=w),
    "residual_norm_bwd": lambda w: _norm_bwd(workspace=w),
}


@pytest.mark.parametrize("name", TAKES)
def test_workspaces_that_hold_less_than_they_count(pools, name):  # noqa: F811
    call = TAKES[name]
    call(T(4096, dtype=U8))
    call(T(1024, dtype=F32))
    for bad in (T(1, dtype=U8).expand(4096), T(8192, dtype=U8)[::2], T(4095, dtype=U8),
                torch.zeros(4096, dtype=U8)):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)


REFUSED = {
    "gated: odd rows of w": (lambda: mx.ragged_gemm_swiglu(T(8, 16), T(2, 47, 16), _ms()), ValueError),
    "gated: w of other columns": (lambda: mx.ragged_gemm_swiglu(T(8, 16), T(2, 48, 8), _ms()), ValueError),
    "gated: w of another type": (lambda: mx.ragged_gemm_swiglu(
        T(8, 16), T(2, 48, 16, dtype=torch.float16), _ms()), ValueError),
    "gated: experts beside splits": (lambda: mx.ragged_gemm_swiglu(T(8, 16), T(3, 48, 16), _ms()), ValueError),
    "gated: fp32": (lambda: mx.ragged_gemm_swiglu(T(8, 16, dtype=F32), T(2, 48, 16, dtype=F32), _ms()),
                    NotImplementedError),
    "gated: strided w": (lambda: mx.ragged_gemm_swiglu(T(8, 16), T(2, 48, 32)[:, :, :16], _ms()), ValueError),
    "gated: strided h": (lambda: mx.ragged_gemm_swiglu(T(8, 16), T(2, 48, 16), _ms(), h=T(8, 64)[:, :48]), ValueError),
    "gated: transposed x": (lambda: mx.ragged_gemm_swiglu(T(16, 8).t(), T(2, 48, 16), _ms()), ValueError),
    "gated: overlapping rows": (lambda: mx.ragged_gemm_swiglu(
        T(64).as_strided((8, 16), (4, 1)), T(2, 48, 16), _ms()), ValueError),
    "gated: row_index of 64 bits": (lambda: mx.ragged_gemm_swiglu(
        T(8, 16), T(2, 48, 16), _ms(), row_index=T(8, dtype=torch.int64)), ValueError),
    "backward: h of other rows": (lambda: mx.ragged_gemm_swiglu_bwd(
        T(8, 24), T(2, 24, 16), T(7, 32), _ms()), ValueError),
    "backward: w of other rows": (lambda: mx.ragged_gemm_swiglu_bwd(
        T(8, 24), T(2, 25, 16), T(8, 32), _ms()), ValueError),
    "fp8: bytes that are not codes": (lambda: mx.ragged_gemm_fp8(
        T(8, 16, dtype=U8), T(8, 1, dtype=F32), T(2, 24, 16, dtype=F8), T(2, 1, 1, dtype=F32), _ms()), ValueError),
    "fp8: scales of other blocks": (lambda: mx.ragged_gemm_fp8(
        T(8, 130, dtype=F8), T(8, 1, dtype=F32), T(2, 24, 130, dtype=F8), T(2, 1, 2, dtype=F32), _ms()), ValueError),
    "fp8: weight scales of other blocks": (lambda: mx.ragged_gemm_fp8(
        T(8, 16, dtype=F8), T(8, 1, dtype=F32), T(2, 130, 16, dtype=F8), T(2, 1, 1, dtype=F32), _ms()), ValueError),
    "fp8: 64-bit results": (lambda: _fp8(out_dtype=torch.float64), NotImplementedError),
    "fp8: weights that are a matrix": (lambda: mx.quantize_fp8_weight(T(8, 16)), ValueError),
    "norm: widths": (lambda: mx.residual_norm(T(6, 8), T(6, 9), pre_weight=T(8, dtype=F32)), ValueError),
    "norm: strided": (lambda: mx.residual_norm(T(6, 16)[:, :8], T(6, 8), pre_weight=T(8, dtype=F32)), ValueError),
    "norm: weights of two types": (lambda: mx.residual_norm(
        T(6, 8), T(6, 8), post_weight=T(8), pre_weight=T(8, dtype=F32)), ValueError),
    "norm: gate of a column": (lambda: mx.residual_norm(
        T(6, 8), T(6, 8), gate=T(6, 1, dtype=F32), pre_weight=T(8, dtype=F32)), ValueError),
    "norm: nothing to do": (lambda: mx.residual_norm(T(6, 8)), ValueError),
    "norm: r without f": (lambda: mx.residual_norm(T(6, 8), pre_weight=T(8, dtype=F32), r=T(6, 8)), ValueError),
    "norm: y without a weight": (lambda: mx.residual_norm(T(6, 8), T(6, 8), y=T(6, 8)), ValueError),
    "norm backward: dy without a weight": (lambda: mx.residual_norm_bwd(T(6, 8), None, T(6, 8), T(6, 8)), ValueError),
    "norm backward: a weight without dy": (lambda: mx.residual_norm_bwd(
        None, T(6, 8), T(6, 8), T(6, 8), pre_weight=T(8, dtype=F32)), ValueError),
    "norm backward: neither": (lambda: mx.residual_norm_bwd(None, None, T(6, 8), T(6, 8)), ValueError),
    "norm backward: dr of another type": (lambda: mx.residual_norm_bwd(
        T(6, 8), T(6, 8), T(6, 8, dtype=F32), T(6, 8), pre_weight=T(8, dtype=F32)), ValueError),
    "norm backward: out of what is not there": (lambda: mx.residual_norm_bwd(
        T(6, 8), None, T(6, 8), T(6, 8), pre_weight=T(8, dtype=F32),
        out=mx.ResidualNormGrad(gate=T(6, dtype=F32))), ValueError),
}


@pytest.mark.parametrize("name", REFUSED)
def test_refused_before_the_library(pools, monkeypatch, name):  # noqa: F811
    call, error = REFUSED[name]

    class Untouched:
        def __getattr__(self, fn):
            assert fn.endswith("_bytes"), fn
            return lambda *args: 0
    with monkeypatch.context() as m:
        m.setattr(binding, "_lib", Untouched)
        with pytest.raises(error):
            call()


def test_fast_sums_of_fp32_results(pools):  # noqa: F811
    with pytest.raises(NotImplementedError):
        _fp8(out_dtype=F32, fast_sums=True)
    assert not pools
    _fp8(fast_sums=True)


def test_norm_backward_leaves_the_given_out_as_it_is(pools):  # noqa: F811
    """Buffers that it lacks are each call's own: a second call writes none of the first one's."""
    x = T(6, 8)
    out = mx.ResidualNormGrad(x=x)
    first, second = _norm_bwd(out=out), _norm_bwd(out=out)
    assert out == mx.ResidualNormGrad(x=x)
    assert first.x is x and second.x is x
    for name in ("f", "gate", "post_weight", "pre_weight"):
        assert getattr(first, name) is not getattr(second, name), name
