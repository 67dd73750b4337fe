"""Which pool the binding's own buffers come from, on the host: nothing here
reaches the library or a GPU.

A block that torch's current stream has freed may still be in use by work queued
there; only calls on that stream are ordered behind it.  So a call that is given
another stream takes its outputs and workspaces from that stream's pool, and
marks the outputs as used by the current stream, where the caller reads them."""

import contextlib

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from moe_expert_grouped_group_amd import binding

BF, F32, U8, I8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int8, torch.int32


class DeviceTensor(torch.Tensor):
    """A host tensor that passes for a device one."""
    is_cuda = True


class Stream:
    def __init__(self, name):
        self.name, self.cuda_stream = name, 64


class Library:
    """Accepts every call; every workspace query asks for room."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("_bytes") else 0


def T(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(DeviceTensor)


@pytest.fixture
def pools(monkeypatch):
    """Records (stream of the pool, streams told of the use) of each buffer."""
    made, current, real = [], [Stream("current")], torch.empty

    def empty(*args, device=None, **kw):
        t = real(*args, **kw).as_subclass(DeviceTensor)
        entry = [current[-1].name, set()]
        t.record_stream = lambda s: entry[1].add(s.name)
        made.append(entry)
        return t

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    binding.ragged_gemm_workspace_bytes.cache_clear()
    binding.moe_route_workspace_bytes.cache_clear()
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", empty)
        m.setattr(torch.cuda, "stream", on)
        m.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
        m.setattr(binding, "_lib", Library)
        m.setattr(binding, "_stream", lambda s: 0)
        yield made
    binding.ragged_gemm_workspace_bytes.cache_clear()
    binding.moe_route_workspace_bytes.cache_clear()


def _ms():
    return T(2, dtype=torch.int64)


def _route():
    return mx.Route(T(6, 2, dtype=I32), T(6, 2, dtype=F32), T(4, dtype=torch.int64), T(12, dtype=I32),
                    T(6, 2, dtype=I32))


# call, buffers that it returns, workspaces that it makes
CALLS = {
    "ragged_gemm NT": (lambda s: mx.ragged_gemm("NT", T(8, 16), T(2, 24, 16), _ms(), stream=s), 1, 1),
    "ragged_gemm NN": (lambda s: mx.ragged_gemm("NN", T(8, 24), T(2, 24, 16), _ms(), stream=s), 1, 1),
    "ragged_gemm TN": (lambda s: mx.ragged_gemm("TN", T(8, 24), T(8, 16), _ms(), stream=s), 1, 1),
    "quantize_int8": (lambda s: mx.quantize_int8(T(8, 16), stream=s), 2, 0),
    "ragged_gemm_int8": (lambda s: mx.ragged_gemm_int8(
        T(8, 16, dtype=I8), T(8, dtype=F32), T(2, 24, 16, dtype=I8), T(2, 24, dtype=F32), _ms(), stream=s), 1, 1),
    "moe_route": (lambda s: mx.moe_route(T(6, 4, dtype=F32), 2, stream=s), 5, 1),
    "moe_route_bwd": (lambda s: mx.moe_route_bwd(T(6, 4, dtype=F32), _route(), T(6, 2, dtype=F32), stream=s), 1, 0),
    "moe_combine": (lambda s: mx.moe_combine(T(12, 8), T(6, 2, dtype=I32), stream=s), 1, 0),
    "moe_combine_bwd": (lambda s: mx.moe_combine_bwd(T(6, 8), T(12, 8), T(6, 2, dtype=I32), stream=s), 2, 0),
    "group_quantize": (lambda s: mx.group_quantize(T(128, 512), usage=3, stream=s), 4, 0),
    "swiglu_quantize": (lambda s: mx.swiglu_quantize(T(128, 1024), stream=s), 4, 0),
    "requant_colwise": (lambda s: mx.requant_colwise(
        T(128, 512, dtype=U8), T(128, 16, dtype=U8), _ms(), with_dbias=True, stream=s), 3, 1),
    "group_quantize_requant": (lambda s: mx.group_quantize_requant(
        T(128, 512), _ms(), with_dbias=True, stream=s), 5, 1),
    "group_quantize_requant_noalloc": (lambda s: mx.group_quantize_requant_noalloc(
        T(128, 512), _ms(), with_dbias=True, stream=s), 5, 0),
    "grouped_dbias": (lambda s: mx.grouped_dbias(
        T(128, 512, dtype=U8), T(128, 16, dtype=U8), _ms(), stream=s), 1, 1),
    "grouped_scaled_bias_grad": (lambda s: mx.grouped_scaled_bias_grad(
        T(128, 512, dtype=U8), T(128, 16, dtype=U8), _ms(), T(128, dtype=F32), T(2, 512, dtype=F32), stream=s), 2, 1),
    "grouped_gemm": (lambda s: mx.grouped_gemm(
        "NT", T(128, 512, dtype=U8), T(128, 16, dtype=U8), T(1024, 512, dtype=U8), T(1024, 16, dtype=U8), _ms(),
        128, 512, 512, stream=s), 1, 0),
    "grouped_gemm_swiglu_quantize": (lambda s: mx.grouped_gemm_swiglu_quantize(
        T(128, 512, dtype=U8), T(128, 16, dtype=U8), T(2048, 512, dtype=U8), T(2048, 16, dtype=U8), _ms(),
        128, 512, 512, stream=s), 5, 0),
    "validate_splits": (lambda s: mx.validate_splits(_ms(), 128, stream=s), 1, 0),
    "swiglu_fwd": (lambda s: mx.swiglu_fwd(T(128, 1024), stream=s), 1, 0),
    "swiglu_bwd_quantize": (lambda s: mx.swiglu_bwd_quantize(
        T(128, 1024), T(128, 512), _ms(), with_dbias=True, stream=s), 5, 1),
    "swiglu_bwd": (lambda s: mx.swiglu_bwd(T(128, 1024), T(128, 512), stream=s), 1, 0),
    "convert_sweep": (lambda s: mx.convert_sweep(0, stream=s), 1, 0),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_given_stream(pools, name):
    call, returned, scratch = CALLS[name]
    call(Stream("given"))
    assert len(pools) == returned + scratch
    assert {pool for pool, _ in pools} == {"given"}
    assert sum(told == {"current"} for _, told in pools) >= returned


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_current_stream(pools, name):
    call, returned, scratch = CALLS[name]
    call(None)
    assert len(pools) == returned + scratch
    assert {pool for pool, _ in pools} == {"current"}


# calls that take a workspace
TAKES = {
    "ragged_gemm": lambda w: mx.ragged_gemm("NN", T(8, 24), T(2, 24, 16), _ms(), workspace=w),
    "ragged_gemm_int8": lambda w: mx.ragged_gemm_int8(
        T(8, 16, dtype=I8), T(8, dtype=F32), T(2, 24, 16, dtype=I8), T(2, 24, dtype=F32), _ms(), workspace=w),
    "moe_route": lambda w: mx.moe_route(T(6, 4, dtype=F32), 2, workspace=w),
    "requant_colwise": lambda w: mx.requant_colwise(
        T(128, 512, dtype=U8), T(128, 16, dtype=U8), _ms(), with_dbias=True, workspace=w),
    "group_quantize_requant": lambda w: mx.group_quantize_requant(
        T(128, 512), _ms(), with_dbias=True, workspace=w),
    "grouped_dbias": lambda w: mx.grouped_dbias(
        T(128, 512, dtype=U8), T(128, 16, dtype=U8), _ms(), workspace=w),
    "grouped_scaled_bias_grad": lambda w: mx.grouped_scaled_bias_grad(
        T(128, 512, dtype=U8), T(128, 16, dtype=U8), _ms(), T(128, dtype=F32), T(2, 512, dtype=F32), workspace=w),
    "swiglu_bwd_quantize": lambda w: mx.swiglu_bwd_quantize(
        T(128, 1024), T(128, 512), _ms(), with_dbias=True, workspace=w),
    "grouped_gemm": lambda w: mx.grouped_gemm(
        "NT", T(128, 512, dtype=U8), T(128, 16, dtype=U8), T(1024, 512, dtype=U8), T(1024, 16, dtype=U8), _ms(),
        128, 512, 512, workspace=w),
    "grouped_gemm_wgrad_accumulate": lambda w: mx.grouped_gemm_wgrad_accumulate(
        T(512, 128, dtype=U8), T(512, 4, dtype=U8), T(512, 128, dtype=U8), T(512, 4, dtype=U8), _ms(), 128, 512, 512,
        T(2, 512, 512, dtype=F32), workspace=w),
}


@pytest.mark.parametrize("name", TAKES)
def test_workspaces_that_hold_less_than_they_count(pools, name):
    """A workspace is `numel` elements from its pointer on: a view that lies on fewer or
    on others is refused, as are a host buffer and one too short."""
    call = TAKES[name]
    call(T(4096, dtype=U8))
    call(T(1024, dtype=F32))
    for bad in (T(1, dtype=U8).expand(4096), T(8192, dtype=U8)[::2], T(4095, dtype=U8),
                torch.zeros(4096, dtype=U8)):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)


@pytest.mark.parametrize("top_k", [-1, 0, 5, 17, 1 << 40])
def test_route_refuses_top_k_before_it_allocates(pools, top_k):
    """The outputs' sizes go by top_k: a ValueError, not the allocator's error or its memory."""
    with pytest.raises(ValueError, match="top_k"):
        mx.moe_route(T(6, 4, dtype=F32), top_k)
    with pytest.raises(ValueError, match="top_k"):
        mx.moe_route(T(6, 40, dtype=F32), top_k if top_k != 5 else 41)
    assert not pools
