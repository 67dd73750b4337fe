"""Thin Python binding of the C ABI (include/mxfp8moe.h).

Argument marshalling only: shapes and dtypes are checked, outputs are
allocated with torch when the caller does not pass them, and every step of
the computation runs in the HIP kernels of libmxfp8moe.so on the current
torch stream (or the stream given, from whose pool its buffers then come; the
caller orders that stream behind the inputs and ahead of the results' use).
The entry points have the C names without the ``mxfp8_`` prefix.
"""

import contextlib
import functools
from dataclasses import dataclass
from typing import Optional

import torch

from . import _native

ROWWISE = 1
COLWISE = 2
LAYOUT_NT, LAYOUT_NN, LAYOUT_TN = 0, 1, 2
_LAYOUTS = {"NT": LAYOUT_NT, "NN": LAYOUT_NN, "TN": LAYOUT_TN, 0: 0, 1: 1, 2: 2}
_OUT = {torch.float32: 0, torch.bfloat16: 1}


@dataclass
class MXFP8Tensor:
    """Row-wise and/or column-wise MXFP8 copies of a [T, K] tensor.

    row_data [T, K] u8 + row_scale [T, K/32] u8; col_data [K, T] u8 +
    col_scale [K, T/32] u8 (the column-wise copy stored transposed).
    """
    row_data: Optional[torch.Tensor] = None
    row_scale: Optional[torch.Tensor] = None
    col_data: Optional[torch.Tensor] = None
    col_scale: Optional[torch.Tensor] = None


def _lib():
    return _native.load()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The raw stream: the one given, or torch's current one (without making
    the stream object, which costs as much as a launch)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t, dtype, shape, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _pool(stream):
    """The context in which memory comes from the pool of the stream that will use
    it.  A block of another stream's pool may still be in use by work queued
    there, which nothing here is ordered behind."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    """An output that this call allocates.  The caller reads it on the current
    stream, which the allocator is told."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    reader = torch.cuda.current_stream(device)
    with _pool(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(reader)
    return t


def _scratch(size, device, stream):
    """A workspace for this call alone: only `stream` ever uses it."""
    with _pool(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _sized(workspace, need):
    """The bytes of a caller's workspace: the kernels write `need` from its pointer on."""
    size = workspace.numel() * workspace.element_size()
    if not workspace.is_cuda or not workspace.is_contiguous() or size < need:
        raise ValueError(f"workspace must be a contiguous device buffer of at least {need} bytes")
    return size


def _as_shape(t, shape, name):
    """View a contiguous u8 operand with the expected number of bytes as `shape`."""
    n = 1
    for d in shape:
        n *= d
    if t.numel() != n:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    t = t.view(shape)
    _need(t, torch.uint8, shape, name)
    return t


def _splits(m_splits, name="m_splits"):
    if not isinstance(m_splits, torch.Tensor) or not m_splits.is_cuda or m_splits.dtype != torch.int64:
        raise ValueError(f"{name} must be a device int64 tensor")
    if not m_splits.is_contiguous() or m_splits.dim() != 1:
        raise ValueError(f"{name} must be a contiguous 1-D tensor")
    return m_splits


def _mx_outputs(out, usage, t, k, like, stream):
    """Allocate (or check) the requested row-/column-wise buffers of a [t, k] tensor."""
    out = out or MXFP8Tensor()
    if usage & ROWWISE:
        if out.row_data is None:
            out.row_data = _empty((t, k), torch.uint8, like.device, stream)
            out.row_scale = _empty((t, k // 32), torch.uint8, like.device, stream)
        _need(out.row_data, torch.uint8, (t, k), "row_data")
        _need(out.row_scale, torch.uint8, (t, k // 32), "row_scale")
    if usage & COLWISE:
        if out.col_data is None:
            out.col_data = _empty((k, t), torch.uint8, like.device, stream)
            out.col_scale = _empty((k, t // 32), torch.uint8, like.device, stream)
        _need(out.col_data, torch.uint8, (k, t), "col_data")
        _need(out.col_scale, torch.uint8, (k, t // 32), "col_scale")
    return out


def _mx_ptrs(out, usage):
    row = usage & ROWWISE
    col = usage & COLWISE
    return (_ptr(out.row_data) if row else None, _ptr(out.row_scale) if row else None,
            _ptr(out.col_data) if col else None, _ptr(out.col_scale) if col else None)


def group_quantize(x, usage=ROWWISE, out: Optional[MXFP8Tensor] = None, noop_flag=None,
                   stream=None):
    """bf16 [T, K] (or [G, N, K], taken as [G*N, K]) -> MXFP8Tensor.

    noop_flag: optional device int32 [1]; when it holds a non-zero value as
    the kernels run, nothing is written and `out` keeps its contents.
    """
    lib = _lib()
    if x.dim() != 2:
        with _pool(stream):   # a copy, where it takes one, is made and used on one stream
            x = x.reshape(-1, x.shape[-1])
    t, k = x.shape
    _need(x, torch.bfloat16, (t, k), "x")
    out = _mx_outputs(out, usage, t, k, x, stream)
    if noop_flag is not None:
        _need(noop_flag, torch.int32, (1,), "noop_flag")
    st = lib.mxfp8_group_quantize(_ptr(x), t, k, usage, *_mx_ptrs(out, usage), _ptr(noop_flag),
                                  _stream(stream))
    _native.check(st, "mxfp8_group_quantize")
    return out


def swiglu_quantize(h, usage=ROWWISE | COLWISE, out: Optional[MXFP8Tensor] = None,
                    stream=None):
    """h [T, 2F] bf16 -> MXFP8Tensor of a = silu(h[:, :F]) * h[:, F:] (bf16
    rounded, as swiglu_fwd gives it) without writing a."""
    lib = _lib()
    t, f2 = h.shape
    f = f2 // 2
    _need(h, torch.bfloat16, (t, 2 * f), "h")
    out = _mx_outputs(out, usage, t, f, h, stream)
    st = lib.mxfp8_swiglu_quantize(_ptr(h), t, f, usage, *_mx_ptrs(out, usage), _stream(stream))
    _native.check(st, "mxfp8_swiglu_quantize")
    return out


def dbias_workspace_bytes(t, n):
    return int(_lib().mxfp8_dbias_workspace_bytes(t, n))


def _workspace(t, n, like, workspace, stream):
    need = dbias_workspace_bytes(t, n)
    if workspace is None:
        workspace = _scratch(max(need, 1), like.device, stream)
    _sized(workspace, need)
    return workspace


def requant_colwise(row_data, row_scale, m_splits=None, with_dbias=False, out=None,
                    dbias=None, workspace=None, stream=None):
    """Row-wise MXFP8 [T, K] -> column-wise copy ([K, T], [K, T/32]) (+ dbias [G, K])."""
    lib = _lib()
    t, k = row_data.shape
    _need(row_data, torch.uint8, (t, k), "row_data")
    _need(row_scale, torch.uint8, (t, k // 32), "row_scale")
    out = out or MXFP8Tensor(row_data=row_data, row_scale=row_scale)
    if out.col_data is None:
        out.col_data = _empty((k, t), torch.uint8, row_data.device, stream)
        out.col_scale = _empty((k, t // 32), torch.uint8, row_data.device, stream)
    _need(out.col_data, torch.uint8, (k, t), "col_data")
    _need(out.col_scale, torch.uint8, (k, t // 32), "col_scale")
    g = 0
    ms = None
    if with_dbias:
        ms = _splits(m_splits)
        g = ms.numel()
        if dbias is None:
            dbias = _empty((g, k), torch.float32, row_data.device, stream)
        _need(dbias, torch.float32, (g, k), "dbias")
        workspace = _workspace(t, k, row_data, workspace, stream)
    st = lib.mxfp8_requant_colwise(
        _ptr(row_data), _ptr(row_scale), t, k, _ptr(out.col_data), _ptr(out.col_scale),
        _ptr(ms), g, _ptr(dbias) if with_dbias else None,
        _ptr(workspace) if with_dbias else None,
        workspace.numel() * workspace.element_size() if with_dbias else 0, _stream(stream))
    _native.check(st, "mxfp8_requant_colwise")
    return (out, dbias) if with_dbias else out


def group_quantize_requant(x, m_splits=None, with_dbias=False, out=None, dbias=None,
                           workspace=None, stream=None):
    """bf16 [T, K] -> MXFP8Tensor with the row-wise copy and the column-wise
    copy requantized from it (+ dbias [G, K] from the dequantized row-wise
    values), in one pass: the bytes of group_quantize(ROWWISE) followed by
    requant_colwise.  Returns the tensor, or (tensor, dbias) with_dbias."""
    lib = _lib()
    t, k = x.shape
    _need(x, torch.bfloat16, (t, k), "x")
    out = _mx_outputs(out, ROWWISE | COLWISE, t, k, x, stream)
    g = 0
    ms = None
    if with_dbias:
        ms = _splits(m_splits)
        g = ms.numel()
        if dbias is None:
            dbias = _empty((g, k), torch.float32, x.device, stream)
        _need(dbias, torch.float32, (g, k), "dbias")
        workspace = _workspace(t, k, x, workspace, stream)
    st = lib.mxfp8_group_quantize_requant(
        _ptr(x), t, k, _ptr(out.row_data), _ptr(out.row_scale), _ptr(out.col_data),
        _ptr(out.col_scale), _ptr(ms), g, _ptr(dbias) if with_dbias else None,
        _ptr(workspace) if with_dbias else None,
        workspace.numel() * workspace.element_size() if with_dbias else 0, _stream(stream))
    _native.check(st, "mxfp8_group_quantize_requant")
    return (out, dbias) if with_dbias else out


NOALLOC_SCRATCH_BYTES = 32 << 20   # MXFP8_NOALLOC_SCRATCH_BYTES of the C header


def group_quantize_requant_noalloc(x, m_splits=None, with_dbias=False, out=None, dbias=None,
                                   stream=None):
    """group_quantize_requant without a workspace: the dbias partial sums go
    to the library's static per-GPU scratch (mxfp8_group_quantize_requant_
    noalloc; with dbias, (T/128) * K * 4 <= NOALLOC_SCRATCH_BYTES).  Calls
    with dbias that overlap on one GPU race on that scratch.  Pass `out` (and
    `dbias`) to keep the call free of allocations."""
    lib = _lib()
    t, k = x.shape
    _need(x, torch.bfloat16, (t, k), "x")
    out = _mx_outputs(out, ROWWISE | COLWISE, t, k, x, stream)
    g = 0
    ms = None
    if with_dbias:
        ms = _splits(m_splits)
        g = ms.numel()
        if dbias is None:
            dbias = _empty((g, k), torch.float32, x.device, stream)
        _need(dbias, torch.float32, (g, k), "dbias")
    st = lib.mxfp8_group_quantize_requant_noalloc(
        _ptr(x), t, k, _ptr(out.row_data), _ptr(out.row_scale), _ptr(out.col_data),
        _ptr(out.col_scale), _ptr(ms), g, _ptr(dbias) if with_dbias else None, _stream(stream))
    _native.check(st, "mxfp8_group_quantize_requant_noalloc")
    return (out, dbias) if with_dbias else out


def grouped_dbias(row_data, row_scale, m_splits, dbias=None, workspace=None, stream=None):
    """Row-wise MXFP8 dY [T, N] -> dbias [G, N] fp32 (sum over each expert's rows)."""
    lib = _lib()
    t, n = row_data.shape
    _need(row_data, torch.uint8, (t, n), "row_data")
    _need(row_scale, torch.uint8, (t, n // 32), "row_scale")
    ms = _splits(m_splits)
    g = ms.numel()
    if dbias is None:
        dbias = _empty((g, n), torch.float32, row_data.device, stream)
    _need(dbias, torch.float32, (g, n), "dbias")
    workspace = _workspace(t, n, row_data, workspace, stream)
    st = lib.mxfp8_grouped_dbias(_ptr(row_data), _ptr(row_scale), t, n, _ptr(ms), g,
                                 _ptr(dbias), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    _native.check(st, "mxfp8_grouped_dbias")
    return dbias


def grouped_scaled_bias_grad(row_data, row_scale, m_splits, scales=None, bias=None,
                             want_dbias=True, want_dscales=True, workspace=None, out=None,
                             stream=None):
    """Gradients of a routing-scaled bias from row-wise MXFP8 dY [T, N]:
    dbias [G, N] = sum over each expert's rows of scales[r] dY[r] (needs
    scales [T] fp32) and dscales [T] = dY[r] . bias[g] (needs bias [G, N]
    fp32).  out: optional (dbias, dscales) buffers to write into.  Returns
    (dbias or None, dscales or None)."""
    lib = _lib()
    t, n = row_data.shape
    _need(row_data, torch.uint8, (t, n), "row_data")
    _need(row_scale, torch.uint8, (t, n // 32), "row_scale")
    ms = _splits(m_splits)
    g = ms.numel()
    dbias, dscales = (None, None) if out is None else out
    if want_dbias:
        _need(scales, torch.float32, (t,), "scales")
        dbias = _empty((g, n), torch.float32, row_data.device, stream) if dbias is None else dbias
        _need(dbias, torch.float32, (g, n), "dbias")
    else:
        dbias = None
    if want_dscales:
        _need(bias, torch.float32, (g, n), "bias")
        if dscales is None:
            dscales = _empty((t,), torch.float32, row_data.device, stream)
        _need(dscales, torch.float32, (t,), "dscales")
    else:
        dscales = None
    need = lib.mxfp8_scaled_bias_workspace_bytes(t, n)
    if workspace is None:
        workspace = _scratch(max(need, 1), row_data.device, stream)
    _sized(workspace, need)
    st = lib.mxfp8_grouped_scaled_bias_grad(
        _ptr(row_data), _ptr(row_scale), t, n, _ptr(ms), g, _ptr(scales) if want_dbias else None,
        _ptr(bias) if want_dscales else None, _ptr(dbias), _ptr(dscales), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _native.check(st, "mxfp8_grouped_scaled_bias_grad")
    return dbias, dscales


def gemm_workspace_bytes():
    return int(_lib().mxfp8_grouped_gemm_workspace_bytes())


def _gemm_workspace(workspace):
    _sized(workspace, gemm_workspace_bytes())
    return workspace


def grouped_gemm(layout, a_data, a_scale, b_data, b_scale, m_splits, tokens, n, k,
                 out_dtype=torch.float32, out=None, stream=None, workspace=None):
    """One grouped GEMM of an expert linear (in_features k, out_features n).

    layout "NT" (forward): a = X row-wise [T, k], b = W row-wise [G, n, k] -> [T, n]
    layout "NN" (dgrad):   a = dY row-wise [T, n], b = W column-wise [k, G*n] -> [T, k]
    layout "TN" (wgrad):   a = dY column-wise [n, T], b = X column-wise [k, T] -> [G, n, k]

    workspace: optional device buffer of gemm_workspace_bytes(); with it the
    wgrad tiles are handed out dynamically (mxfp8_grouped_gemm_ws), same bytes.
    """
    lib = _lib()
    lay = _LAYOUTS[layout]
    ms = _splits(m_splits)
    g = ms.numel()
    t = tokens
    if out_dtype not in _OUT:
        raise NotImplementedError(f"output dtype {out_dtype} is not supported")
    if lay == LAYOUT_NT:
        shapes = ((t, k), (t, k // 32), (g * n, k), (g * n, k // 32), (t, n))
    elif lay == LAYOUT_NN:
        shapes = ((t, n), (t, n // 32), (k, g * n), (k, g * n // 32), (t, k))
    else:
        shapes = ((n, t), (n, t // 32), (k, t), (k, t // 32), (g, n, k))
    a2 = _as_shape(a_data, shapes[0], "a_data")
    as2 = _as_shape(a_scale, shapes[1], "a_scale")
    b2 = _as_shape(b_data, shapes[2], "b_data")
    bs2 = _as_shape(b_scale, shapes[3], "b_scale")
    if out is None:
        out = _empty(shapes[4], out_dtype, a2.device, stream)
    _need(out, out_dtype, shapes[4], "out")
    if workspace is None:
        st = lib.mxfp8_grouped_gemm(lay, _ptr(a2), _ptr(as2), _ptr(b2), _ptr(bs2), _ptr(out),
                                    _OUT[out_dtype], t, n, k, _ptr(ms), g, _stream(stream))
        _native.check(st, "mxfp8_grouped_gemm")
    else:
        ws = _gemm_workspace(workspace)
        st = lib.mxfp8_grouped_gemm_ws(lay, _ptr(a2), _ptr(as2), _ptr(b2), _ptr(bs2), _ptr(out),
                                       _OUT[out_dtype], t, n, k, _ptr(ms), g, _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream(stream))
        _native.check(st, "mxfp8_grouped_gemm_ws")
    return out


def grouped_gemm_swiglu_quantize(a_data, a_scale, b_data, b_scale, m_splits, tokens, f, k,
                                 usage=ROWWISE | COLWISE, h=None, out=None, stream=None):
    """Forward of the fused MLP's FC1 with SwiGLU + quantize in the epilogue:
    h [T, 2F] = X W1_g^T (bf16; a = X row-wise [T, k], b = W1 row-wise
    [G, 2F, k]) and the MXFP8Tensor of a = silu(h[:, :F]) * h[:, F:] (the
    bytes of grouped_gemm + swiglu_quantize).  Returns (h, MXFP8Tensor)."""
    lib = _lib()
    ms = _splits(m_splits)
    g = ms.numel()
    t = tokens
    a2 = _as_shape(a_data, (t, k), "a_data")
    as2 = _as_shape(a_scale, (t, k // 32), "a_scale")
    b2 = _as_shape(b_data, (g * 2 * f, k), "b_data")
    bs2 = _as_shape(b_scale, (g * 2 * f, k // 32), "b_scale")
    if h is None:
        h = _empty((t, 2 * f), torch.bfloat16, a2.device, stream)
    _need(h, torch.bfloat16, (t, 2 * f), "h")
    out = _mx_outputs(out, usage, t, f, a2, stream)
    st = lib.mxfp8_grouped_gemm_swiglu_quantize(
        _ptr(a2), _ptr(as2), _ptr(b2), _ptr(bs2), _ptr(h), t, f, k, _ptr(ms), g, usage,
        *_mx_ptrs(out, usage), _stream(stream))
    _native.check(st, "mxfp8_grouped_gemm_swiglu_quantize")
    return h, out


def grouped_gemm_wgrad_accumulate(a_data, a_scale, b_data, b_scale, m_splits, tokens, n, k,
                                  main_grad, stream=None, workspace=None):
    """wgrad added into an fp32 main_grad [G, n, k] in place:
    main_grad[g] += dY_g^T X_g (a = dY column-wise [n, T], b = X column-wise
    [k, T]); experts without tokens keep their main_grad untouched."""
    lib = _lib()
    ms = _splits(m_splits)
    g = ms.numel()
    t = tokens
    a2 = _as_shape(a_data, (n, t), "a_data")
    as2 = _as_shape(a_scale, (n, t // 32), "a_scale")
    b2 = _as_shape(b_data, (k, t), "b_data")
    bs2 = _as_shape(b_scale, (k, t // 32), "b_scale")
    _need(main_grad, torch.float32, (g, n, k), "main_grad")
    if workspace is None:
        st = lib.mxfp8_grouped_gemm_wgrad_accumulate(_ptr(a2), _ptr(as2), _ptr(b2), _ptr(bs2),
                                                     _ptr(main_grad), t, n, k, _ptr(ms), g,
                                                     _stream(stream))
        _native.check(st, "mxfp8_grouped_gemm_wgrad_accumulate")
    else:
        ws = _gemm_workspace(workspace)
        st = lib.mxfp8_grouped_gemm_wgrad_accumulate_ws(
            _ptr(a2), _ptr(as2), _ptr(b2), _ptr(bs2), _ptr(main_grad), t, n, k, _ptr(ms), g,
            _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
        _native.check(st, "mxfp8_grouped_gemm_wgrad_accumulate_ws")
    return main_grad


def validate_splits(m_splits, tokens, flag=None, stream=None):
    """Enqueue the device-side split check; returns the device int32 flag tensor."""
    lib = _lib()
    ms = _splits(m_splits)
    if flag is None:
        flag = _empty((1,), torch.int32, ms.device, stream)
    st = lib.mxfp8_validate_splits(_ptr(ms), ms.numel(), tokens, _ptr(flag), _stream(stream))
    _native.check(st, "mxfp8_validate_splits")
    return flag


def swiglu_fwd(h, out=None, stream=None):
    """h [T, 2F] bf16 -> silu(h[:, :F]) * h[:, F:] as bf16 [T, F]."""
    lib = _lib()
    t, f2 = h.shape
    f = f2 // 2
    _need(h, torch.bfloat16, (t, 2 * f), "h")
    if out is None:
        out = _empty((t, f), torch.bfloat16, h.device, stream)
    _need(out, torch.bfloat16, (t, f), "out")
    _native.check(lib.mxfp8_swiglu_fwd(_ptr(h), t, f, _ptr(out), _stream(stream)),
                  "mxfp8_swiglu_fwd")
    return out


def swiglu_bwd_quantize(h, da, m_splits=None, with_dbias=False, out=None, dbias=None,
                        workspace=None, stream=None):
    """SwiGLU backward of h [T, 2F] and da [T, F] (bf16) quantized as
    group_quantize_requant quantizes dh [T, 2F], without writing dh: the bytes
    (and dbias [G, 2F]) of swiglu_bwd followed by group_quantize_requant.
    Returns the tensor, or (tensor, dbias) with_dbias."""
    lib = _lib()
    t, k = h.shape
    f = k // 2
    _need(h, torch.bfloat16, (t, 2 * f), "h")
    _need(da, torch.bfloat16, (t, f), "da")
    out = _mx_outputs(out, ROWWISE | COLWISE, t, k, h, stream)
    g = 0
    ms = None
    if with_dbias:
        ms = _splits(m_splits)
        g = ms.numel()
        if dbias is None:
            dbias = _empty((g, k), torch.float32, h.device, stream)
        _need(dbias, torch.float32, (g, k), "dbias")
        workspace = _workspace(t, k, h, workspace, stream)
    st = lib.mxfp8_swiglu_bwd_quantize(
        _ptr(h), _ptr(da), t, f, _ptr(out.row_data), _ptr(out.row_scale), _ptr(out.col_data),
        _ptr(out.col_scale), _ptr(ms), g, _ptr(dbias) if with_dbias else None,
        _ptr(workspace) if with_dbias else None,
        workspace.numel() * workspace.element_size() if with_dbias else 0, _stream(stream))
    _native.check(st, "mxfp8_swiglu_bwd_quantize")
    return (out, dbias) if with_dbias else out


def swiglu_bwd(h, da, out=None, stream=None):
    """Gradient of swiglu_fwd w.r.t. h, given da [T, F]; returns bf16 [T, 2F]."""
    lib = _lib()
    t, f2 = h.shape
    f = f2 // 2
    _need(h, torch.bfloat16, (t, 2 * f), "h")
    _need(da, torch.bfloat16, (t, f), "da")
    if out is None:
        out = _empty((t, 2 * f), torch.bfloat16, h.device, stream)
    _need(out, torch.bfloat16, (t, 2 * f), "out")
    _native.check(lib.mxfp8_swiglu_bwd(_ptr(h), _ptr(da), t, f, _ptr(out), _stream(stream)),
                  "mxfp8_swiglu_bwd")
    return out


def convert_sweep(mode, stream=None):
    """Diagnostic: the device conversion helpers over every (value, scale byte)
    pair (layouts in mxfp8_convert_sweep's header comment); a uint8 tensor."""
    lib = _lib()
    need = lib.mxfp8_convert_sweep_bytes(mode)
    if need == 0:
        raise ValueError(f"unknown sweep mode {mode}")
    out = _empty((need,), torch.uint8, torch.device("cuda"), stream)
    st = lib.mxfp8_convert_sweep(mode, _ptr(out), need, _stream(stream))
    _native.check(st, "mxfp8_convert_sweep")
    return out


# ----------------------------------------------------------------------------
# experts with any number of rows, and the routing around them
# ----------------------------------------------------------------------------

_TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _rows_of(t, dtype, shape, name):
    """A device matrix with contiguous rows; returns its row stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    ld = t.stride(0) if shape[0] > 1 else shape[1]
    if ld < shape[1]:
        raise ValueError(f"{name} must not have overlapping rows")
    return ld


def _matrix(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    return t.shape


def _type_of(t, name, floats=(torch.bfloat16, torch.float16)):
    if t.dtype not in floats:
        raise NotImplementedError(f"{name} of {t.dtype} is not supported")
    return _TYPE[t.dtype]


def _same_device(like, **tensors):
    at = like.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != at:
            raise ValueError(f"{name} is on {t.device}, not on {like.device}")


def _row_index(row_index, like):
    if row_index is None:
        return None
    if not isinstance(row_index, torch.Tensor) or row_index.dim() != 1:
        raise ValueError("row_index must be a 1-D tensor")
    _need(row_index, torch.int32, tuple(row_index.shape), "row_index")
    return row_index


@functools.lru_cache(maxsize=4096)
def ragged_gemm_workspace_bytes(layout, dtype, rows, x_rows, n, k, groups):
    """Workspace of ragged_gemm (bf16, fp16) or ragged_gemm_int8 (int8, "NT")
    for these sizes; 0 where none is used."""
    return int(_lib().mxfp8_ragged_gemm_workspace_bytes(_LAYOUTS[layout], dtype.itemsize, rows,
                                                        x_rows, n, k, groups))


def _ragged_workspace(workspace, like, stream, *sizes):
    """(buffer, its bytes): the caller's, or one for this call (torch's
    allocator hands the same memory out again)."""
    need = ragged_gemm_workspace_bytes(*sizes)
    if workspace is None:
        if need == 0:
            return None, 0
        return _scratch(need, like.device, stream), need
    return workspace, _sized(workspace, need)


def ragged_gemm(layout, a, b, m_splits, row_index=None, out_dtype=None, out=None, stream=None,
                workspace=None):
    """One product of an expert linear whose experts have any number of rows.

    layout "NT" (forward): a = X [S, K], b = W [G, N, K] -> [R, N]
    layout "NN" (dgrad):   a = dY [R, N], b = W [G, N, K] -> [R, K]
    layout "TN" (wgrad):   a = dY [R, N], b = X [S, K] -> [G, N, K]

    bf16 or fp16 operands; m_splits device int64 [G], expert g owning that many
    consecutive rows of R.  row_index (int32 [R], NT and TN): row r of the
    product is row row_index[r] of X; without it S = R.  a, X and out may
    have a row stride.  out_dtype: the operands' (default) or float32.  Rows
    past the last expert's are not written (mxfp8_ragged_gemm).  workspace:
    optional device buffer of ragged_gemm_workspace_bytes(...), not shared by calls
    that may run at the same time; allocated for the call where there is none.
    """
    lib = _lib()
    lay = _LAYOUTS[layout]
    ms = _splits(m_splits)
    g = ms.numel()
    ra, ca = _matrix(a, "a")
    ty = _type_of(a, "a")
    index = _row_index(row_index, a)
    if lay == LAYOUT_TN:
        s, k = _matrix(b, "b")
        r, n = ra, ca
    else:
        if not isinstance(b, torch.Tensor) or b.dim() != 3:
            raise ValueError("b must be [G, N, K]")
        n, k = b.shape[1:]
        s = ra
        r = index.numel() if index is not None and lay == LAYOUT_NT else ra
    if index is not None:
        if lay == LAYOUT_NN:
            raise ValueError("NN takes no row_index")
        if index.numel() != r:
            raise ValueError(f"row_index must have {r} entries, got {index.numel()}")
    elif lay == LAYOUT_TN and s != r:
        raise ValueError(f"b must have {r} rows without a row_index, got {s}")
    lda = _rows_of(a, a.dtype, (ra, k if lay == LAYOUT_NT else n), "a")
    if lay == LAYOUT_TN:
        ldb = _rows_of(b, a.dtype, (s, k), "b")
    else:
        _need(b, a.dtype, (g, n, k), "b")
        ldb = k
    out_dtype = a.dtype if out_dtype is None else out_dtype
    if out_dtype not in (a.dtype, torch.float32):
        raise NotImplementedError(f"output dtype {out_dtype} is not supported")
    if lay == LAYOUT_TN:
        if out is None:
            out = _empty((g, n, k), out_dtype, a.device, stream)
        _need(out, out_dtype, (g, n, k), "out")
        ldc = k
    else:
        shape = (r, n if lay == LAYOUT_NT else k)
        if out is None:
            out = _empty(shape, out_dtype, a.device, stream)
        ldc = _rows_of(out, out_dtype, shape, "out")
    ws, ws_bytes = _ragged_workspace(workspace, a, stream, lay, a.dtype, r, s, n, k, g)
    _same_device(a, b=b, m_splits=ms, row_index=index, out=out, workspace=ws)
    st = lib.mxfp8_ragged_gemm(lay, ty, _ptr(a), lda, _ptr(b), ldb, _ptr(out), ldc,
                               _TYPE[out_dtype], r, s, n, k, _ptr(ms), g, _ptr(index),
                               _ptr(ws), ws_bytes, _stream(stream))
    _native.check(st, "mxfp8_ragged_gemm")
    return out


def quantize_int8(x, out=None, stream=None):
    """Rows of a bf16 / fp16 matrix as 8-bit integers: (q int8 [T, K], scale
    fp32 [T]) with x ~ q * scale, scale = max|row| / 127.  out: optional (q,
    scale) buffers.  For weights [G, N, K] pass the view [G * N, K]."""
    lib = _lib()
    t, k = _matrix(x, "x")
    ty = _type_of(x, "x")
    ldx = _rows_of(x, x.dtype, (t, k), "x")
    q, scale = (None, None) if out is None else out
    q = _empty((t, k), torch.int8, x.device, stream) if q is None else q
    scale = _empty((t,), torch.float32, x.device, stream) if scale is None else scale
    _need(q, torch.int8, (t, k), "q")
    _need(scale, torch.float32, (t,), "scale")
    _same_device(x, q=q, scale=scale)
    st = lib.mxfp8_quantize_int8(_ptr(x), ty, t, k, ldx, _ptr(q), _ptr(scale), _stream(stream))
    _native.check(st, "mxfp8_quantize_int8")
    return q, scale


def ragged_gemm_int8(q, scale, w, w_scale, m_splits, row_index=None, out_dtype=torch.bfloat16,
                     out=None, stream=None, workspace=None):
    """Forward product in 8-bit integers: q [S, K] int8 with scale [S] (as
    quantize_int8 gives them), w [G, N, K] int8 with w_scale [G, N] -> [R, N],
    (sum of q w) * scale * w_scale.  row_index, m_splits and workspace as
    ragged_gemm."""
    lib = _lib()
    ms = _splits(m_splits)
    g = ms.numel()
    s, k = _matrix(q, "q")
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be [G, N, K]")
    n = w.shape[1]
    index = _row_index(row_index, q)
    r = s if index is None else index.numel()
    ldq = _rows_of(q, torch.int8, (s, k), "q")
    _need(scale, torch.float32, (s,), "scale")
    _need(w, torch.int8, (g, n, k), "w")
    _need(w_scale, torch.float32, (g, n), "w_scale")
    if out_dtype not in _TYPE:
        raise NotImplementedError(f"output dtype {out_dtype} is not supported")
    if out is None:
        out = _empty((r, n), out_dtype, q.device, stream)
    ldc = _rows_of(out, out_dtype, (r, n), "out")
    ws, ws_bytes = _ragged_workspace(workspace, q, stream, LAYOUT_NT, torch.int8, r, s, n, k, g)
    _same_device(q, scale=scale, w=w, w_scale=w_scale, m_splits=ms, row_index=index, out=out,
                 workspace=ws)
    st = lib.mxfp8_ragged_gemm_int8(_ptr(q), ldq, _ptr(scale), _ptr(w), _ptr(w_scale), _ptr(out),
                                    ldc, _TYPE[out_dtype], r, s, n, k, _ptr(ms), g, _ptr(index),
                                    _ptr(ws), ws_bytes, _stream(stream))
    _native.check(st, "mxfp8_ragged_gemm_int8")
    return out


@dataclass
class Route:
    """Where the tokens go (moe_route): ids, weights and row_pos [T, top_k],
    m_splits [E], row_token [T * top_k]."""
    ids: torch.Tensor
    weights: torch.Tensor
    m_splits: torch.Tensor
    row_token: torch.Tensor
    row_pos: torch.Tensor
    renormalize: bool = True


@functools.lru_cache(maxsize=256)
def moe_route_workspace_bytes(tokens, experts):
    return int(_lib().mxfp8_moe_route_workspace_bytes(tokens, experts))


def moe_route(logits, top_k, renormalize=True, token_mask=None, out=None, workspace=None,
              stream=None):
    """logits [T, E] (fp32, bf16, fp16) -> Route: each token's top_k experts
    (equal logits by lowest expert) and softmax weights, over the chosen
    experts (renormalize) or over all; the rows' order by expert.  token_mask:
    bool or uint8 [T], tokens with 0 are not routed."""
    lib = _lib()
    t, e = _matrix(logits, "logits")
    ty = _type_of(logits, "logits", tuple(_TYPE))
    _need(logits, logits.dtype, (t, e), "logits")
    if not 1 <= top_k <= min(e, 16):
        raise ValueError(f"top_k = {top_k} must be 1 to min(E, 16)")
    if token_mask is not None:
        if token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        _need(token_mask, torch.uint8, (t,), "token_mask")
    if out is None:
        out = Route(_empty((t, top_k), torch.int32, logits.device, stream),
                    _empty((t, top_k), torch.float32, logits.device, stream),
                    _empty((e,), torch.int64, logits.device, stream),
                    _empty((t * top_k,), torch.int32, logits.device, stream),
                    _empty((t, top_k), torch.int32, logits.device, stream))
    else:
        _need(out.ids, torch.int32, (t, top_k), "ids")
        _need(out.weights, torch.float32, (t, top_k), "weights")
        _need(out.m_splits, torch.int64, (e,), "m_splits")
        _need(out.row_token, torch.int32, (t * top_k,), "row_token")
        _need(out.row_pos, torch.int32, (t, top_k), "row_pos")
    out.renormalize = bool(renormalize)
    need = moe_route_workspace_bytes(t, e)
    size = need
    if workspace is not None:
        size = _sized(workspace, need)
    elif need:
        workspace = _scratch(need, logits.device, stream)
    _same_device(logits, token_mask=token_mask, ids=out.ids, weights=out.weights,
                 m_splits=out.m_splits, row_token=out.row_token, row_pos=out.row_pos,
                 workspace=workspace)
    st = lib.mxfp8_moe_route(_ptr(logits), ty, t, e, top_k, int(out.renormalize),
                             _ptr(token_mask), _ptr(out.ids), _ptr(out.weights),
                             _ptr(out.m_splits), _ptr(out.row_token), _ptr(out.row_pos),
                             _ptr(workspace), size, _stream(stream))
    _native.check(st, "mxfp8_moe_route")
    return out


def moe_route_bwd(logits, route, dweights, out=None, stream=None):
    """Gradient of the logits [T, E] (their type) from that of route.weights."""
    lib = _lib()
    t, e = _matrix(logits, "logits")
    ty = _type_of(logits, "logits", tuple(_TYPE))
    k = _matrix(route.ids, "ids")[1]
    _need(logits, logits.dtype, (t, e), "logits")
    _need(route.ids, torch.int32, (t, k), "ids")
    _need(route.weights, torch.float32, (t, k), "weights")
    _need(dweights, torch.float32, (t, k), "dweights")
    if out is None:
        out = _empty((t, e), logits.dtype, logits.device, stream)
    _need(out, logits.dtype, (t, e), "out")
    _same_device(logits, ids=route.ids, weights=route.weights, dweights=dweights, out=out)
    st = lib.mxfp8_moe_route_bwd(_ptr(logits), ty, t, e, k, int(route.renormalize),
                                 _ptr(route.ids), _ptr(route.weights), _ptr(dweights), _ptr(out),
                                 _stream(stream))
    _native.check(st, "mxfp8_moe_route_bwd")
    return out


def moe_combine(y, row_pos, weights=None, out=None, stream=None):
    """out [T, H] = sum over j of weights[:, j] * y[row_pos[:, j]] (y [R, H]
    bf16 / fp16, fp32 sums).  Without weights the plain sum, which is the
    gradient of the gather by row_token."""
    lib = _lib()
    r, h = _matrix(y, "y")
    ty = _type_of(y, "y")
    t, k = _matrix(row_pos, "row_pos")
    _need(y, y.dtype, (r, h), "y")
    _need(row_pos, torch.int32, (t, k), "row_pos")
    if weights is not None:
        _need(weights, torch.float32, (t, k), "weights")
    if out is None:
        out = _empty((t, h), y.dtype, y.device, stream)
    _need(out, y.dtype, (t, h), "out")
    _same_device(y, row_pos=row_pos, weights=weights, out=out)
    st = lib.mxfp8_moe_combine(_ptr(y), ty, t, r, h, k, _ptr(row_pos), _ptr(weights), _ptr(out),
                               _stream(stream))
    _native.check(st, "mxfp8_moe_combine")
    return out


def moe_combine_bwd(dout, y, row_pos, weights=None, want_dy=True, want_dweights=True, out=None,
                    stream=None):
    """Gradients of moe_combine: (dy [R, H], dweights [T, top_k] fp32), None
    for one that is not wanted.  Rows of dy that no row_pos names are not
    written.  out: optional (dy, dweights) buffers."""
    lib = _lib()
    t, h = _matrix(dout, "dout")
    ty = _type_of(dout, "dout")
    r = _matrix(y, "y")[0]
    k = _matrix(row_pos, "row_pos")[1]
    _need(dout, dout.dtype, (t, h), "dout")
    _need(y, dout.dtype, (r, h), "y")
    _need(row_pos, torch.int32, (t, k), "row_pos")
    if weights is not None:
        _need(weights, torch.float32, (t, k), "weights")
    dy, dw = (None, None) if out is None else out
    if want_dy:
        dy = _empty((r, h), y.dtype, y.device, stream) if dy is None else dy
        _need(dy, dout.dtype, (r, h), "dy")
    else:
        dy = None
    if want_dweights:
        dw = _empty((t, k), torch.float32, dout.device, stream) if dw is None else dw
        _need(dw, torch.float32, (t, k), "dweights")
    else:
        dw = None
    _same_device(dout, y=y, row_pos=row_pos, weights=weights, dy=dy, dweights=dw)
    st = lib.mxfp8_moe_combine_bwd(_ptr(dout), _ptr(y), ty, t, r, h, k, _ptr(row_pos),
                                   _ptr(weights), _ptr(dy), _ptr(dw), _stream(stream))
    _native.check(st, "mxfp8_moe_combine_bwd")
    return dy, dw
