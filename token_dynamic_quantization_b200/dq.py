"""ctypes binding of libdq.so (C ABI in include/dq.h) — argument marshalling only.

The functions named like the C entry points (``dq_get_workspace_size``,
``dq_dynamic_quant``, ``dq_ada_layernorm_quant``, ``dq_status_string``) take
raw integers (device pointers, sizes, enum values, a ``cudaStream_t``) exactly
as the C ABI does. ``dynamic_quant`` and ``ada_layernorm_quant`` are
tensor-level conveniences: they allocate the outputs with torch (device
memory is torch's job here), pass pointers and the current stream, and return
the tensors. Every step of the computation runs in the CUDA kernels.

Importing this module loads the library and raises ImportError if it is
missing; there is no fallback path.
"""

from __future__ import annotations

import ctypes
import functools
import os

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdq.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is not built; run `python -m token_dynamic_quantization_b200.build` "
        "(the CUDA library is required: there is no CPU fallback)")

_lib = ctypes.CDLL(_LIB_PATH)

# ---- enums (values fixed by include/dq.h)
DQ_OK = 0
DQ_ERR_NULL_POINTER = 1
DQ_ERR_BAD_SHAPE = 2
DQ_ERR_BAD_DTYPE = 3
DQ_ERR_UNSUPPORTED = 4
DQ_ERR_MISALIGNED = 5
DQ_ERR_WORKSPACE_TOO_SMALL = 6
DQ_ERR_CUDA = 7
DQ_ERR_BAD_ARGUMENT = 8

DQ_F32, DQ_F16, DQ_BF16, DQ_INT8, DQ_INT4X2, DQ_INT32 = 0, 1, 2, 3, 4, 5
DQ_SYMMETRIC, DQ_ASYMMETRIC = 0, 1
DQ_WS_ROWS_PAST_LAST_GROUP = 0x1
DQ_WS_GROUP_INDEX_INVALID = 0x2
DQ_MAX_GROUPS = 1024
DQ_ADA_NOALLOC_MAX_TABLE = 131072
DQ_ACT_NONE, DQ_ACT_RELU, DQ_ACT_GELU, DQ_ACT_GELU_TANH, DQ_ACT_SILU = 0, 1, 2, 3, 4
DQ_MAX_HEAD_DIM = 256
DQ_MAX_HEADS = 1024

_vp, _i64, _i32, _f32, _sz, _ci = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                                   ctypes.c_size_t, ctypes.c_int)

_lib.dq_status_string.argtypes = [_ci]
_lib.dq_status_string.restype = ctypes.c_char_p
_lib.dq_get_workspace_size.argtypes = [_i64, _i64, _ci, _ci, _ci, _i32, ctypes.POINTER(_sz)]
_lib.dq_get_workspace_size.restype = _ci
_lib.dq_dynamic_quant.argtypes = [_vp, _ci, _i64, _i64, _vp, _ci, _vp, _i32, _ci, _ci, _vp, _vp, _vp, _vp, _sz,
                                  _vp]
_lib.dq_dynamic_quant.restype = _ci
_lib.dq_ada_layernorm_quant_get_workspace_size.argtypes = [_i64, _i64, _i64, _ci, _ci, ctypes.POINTER(_sz)]
_lib.dq_ada_layernorm_quant_get_workspace_size.restype = _ci
_lib.dq_ada_layernorm_quant.argtypes = [_vp, _ci, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _ci, _f32, _vp, _vp,
                                        _vp, _sz, _vp]
_lib.dq_ada_layernorm_quant.restype = _ci
_lib.dq_dequant_per_token.argtypes = [_vp, _ci, _i64, _i64, _vp, _vp, _ci, _vp, _ci, _vp]
_lib.dq_dequant_per_token.restype = _ci
_lib.dq_dequant_per_group.argtypes = [_vp, _ci, _i64, _i64, _vp, _vp, _ci, _i64, _i32, _vp, _ci, _vp]
_lib.dq_dequant_per_group.restype = _ci
_lib.dq_w8a8_gemm.argtypes = [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _ci, _i32, _vp]
_lib.dq_w8a8_gemm.restype = _ci
_lib.dq_ada_layernorm_quant_noalloc.argtypes = [_vp, _ci, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _ci, _f32, _vp,
                                                _vp, _vp]
_lib.dq_ada_layernorm_quant_noalloc.restype = _ci
_lib.dq_w8a8_linear.argtypes = [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _ci, _ci, _vp, _vp, _ci, _vp]
_lib.dq_w8a8_linear.restype = _ci
_lib.dq_qk_norm_rope.argtypes = [_vp, _i64, _vp, _i64, _ci, _i64, _i32, _i32, _i32, _vp, _vp, _ci, _f32, _vp, _vp,
                                 _i32, _i32, _vp, _i64, _vp, _i64, _vp]
_lib.dq_qk_norm_rope.restype = _ci
_lib.dq_qk_norm_rope_cache.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _ci, _i64, _i32, _i32, _i32, _vp, _vp, _ci,
                                       _f32, _vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _ci, _vp, _vp, _vp, _i64,
                                       _i32, _vp]
_lib.dq_qk_norm_rope_cache.restype = _ci
_lib.dq_paged_attention_get_workspace_size.argtypes = [_i64, _i32, _i32, _i32, _ci, ctypes.POINTER(_sz)]
_lib.dq_paged_attention_get_workspace_size.restype = _ci
_lib.dq_paged_attention.argtypes = [_vp, _ci, _i64, _vp, _vp, _ci, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64,
                                    _i32, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _sz, _vp]
_lib.dq_paged_attention.restype = _ci

LIBRARY_PATH = _LIB_PATH


class DQError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(dq_status_string(status))


# ---------------------------------------------------------------- C-ABI mirrors

def dq_status_string(status: int) -> str:
    return _lib.dq_status_string(status).decode()


def dq_get_workspace_size(rows: int, cols: int, x_dtype: int, mode: int, y_dtype: int, num_groups: int) -> int:
    out = _sz(0)
    st = _lib.dq_get_workspace_size(rows, cols, x_dtype, mode, y_dtype, num_groups, ctypes.byref(out))
    if st != DQ_OK:
        raise DQError(st)
    return int(out.value)


def dq_ada_layernorm_quant_get_workspace_size(batch: int, seq: int, hidden: int, x_dtype: int,
                                              param_dtype: int) -> int:
    out = _sz(0)
    st = _lib.dq_ada_layernorm_quant_get_workspace_size(batch, seq, hidden, x_dtype, param_dtype, ctypes.byref(out))
    if st != DQ_OK:
        raise DQError(st)
    return int(out.value)


def dq_dynamic_quant(x, x_dtype, rows, cols, smooth, smooth_dtype, group_index, num_groups, mode, y_dtype, y,
                     scale, offset, workspace, workspace_bytes, stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_dynamic_quant(x, x_dtype, rows, cols, smooth, smooth_dtype, group_index, num_groups, mode,
                                 y_dtype, y, scale, offset, workspace, workspace_bytes, stream)


def dq_ada_layernorm_quant(x, x_dtype, batch, seq, hidden, ada_scale, ada_shift, weight, bias, smooth,
                           param_dtype, epsilon, out, quant_scale, workspace, workspace_bytes, stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_ada_layernorm_quant(x, x_dtype, batch, seq, hidden, ada_scale, ada_shift, weight, bias,
                                       smooth, param_dtype, epsilon, out, quant_scale, workspace,
                                       workspace_bytes, stream)


def dq_dequant_per_token(y, y_dtype, rows, cols, scale, offset, scale_dtype, out, out_dtype, stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_dequant_per_token(y, y_dtype, rows, cols, scale, offset, scale_dtype, out, out_dtype, stream)


def dq_dequant_per_group(y, y_dtype, rows, cols, scale, offset, scale_dtype, group_size, k_dim, out, out_dtype,
                         stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_dequant_per_group(y, y_dtype, rows, cols, scale, offset, scale_dtype, group_size, k_dim, out,
                                     out_dtype, stream)


def dq_w8a8_gemm(a, b, m, n, k, a_scale, b_scale, out, out_dtype, accumulate, stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_w8a8_gemm(a, b, m, n, k, a_scale, b_scale, out, out_dtype, accumulate, stream)


def dq_ada_layernorm_quant_noalloc(x, x_dtype, batch, seq, hidden, ada_scale, ada_shift, weight, bias, smooth,
                                   param_dtype, epsilon, out, quant_scale, stream) -> int:
    """Raw call (no workspace: the library's fixed table). Returns the dq_status."""
    return _lib.dq_ada_layernorm_quant_noalloc(x, x_dtype, batch, seq, hidden, ada_scale, ada_shift, weight, bias,
                                               smooth, param_dtype, epsilon, out, quant_scale, stream)


def dq_w8a8_linear(a, b, m, n, k, a_scale, b_scale, bias, bias_dtype, activation, residual, out, out_dtype,
                   stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_w8a8_linear(a, b, m, n, k, a_scale, b_scale, bias, bias_dtype, activation, residual, out,
                               out_dtype, stream)


def dq_qk_norm_rope(q, q_stride, k, k_stride, dtype, tokens, q_heads, kv_heads, head_dim, q_weight, k_weight,
                    weight_dtype, epsilon, positions, inv_freq, rope_dim, interleaved, q_out, q_out_stride, k_out,
                    k_out_stride, stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_qk_norm_rope(q, q_stride, k, k_stride, dtype, tokens, q_heads, kv_heads, head_dim, q_weight,
                                k_weight, weight_dtype, epsilon, positions, inv_freq, rope_dim, interleaved, q_out,
                                q_out_stride, k_out, k_out_stride, stream)


def dq_qk_norm_rope_cache(q, q_stride, k, k_stride, v, v_stride, dtype, tokens, q_heads, kv_heads, head_dim, q_weight,
                          k_weight, weight_dtype, epsilon, positions, inv_freq, rope_dim, interleaved, q_out,
                          q_out_stride, k_cache, v_cache, cache_dtype, k_scale, v_scale, slots, num_pages, page_size,
                          stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_qk_norm_rope_cache(q, q_stride, k, k_stride, v, v_stride, dtype, tokens, q_heads, kv_heads,
                                      head_dim, q_weight, k_weight, weight_dtype, epsilon, positions, inv_freq,
                                      rope_dim, interleaved, q_out, q_out_stride, k_cache, v_cache, cache_dtype,
                                      k_scale, v_scale, slots, num_pages, page_size, stream)


def dq_paged_attention_get_workspace_size(batch: int, q_heads: int, kv_heads: int, head_dim: int,
                                          cache_dtype: int) -> int:
    out = _sz(0)
    st = _lib.dq_paged_attention_get_workspace_size(batch, q_heads, kv_heads, head_dim, cache_dtype,
                                                    ctypes.byref(out))
    if st != DQ_OK:
        raise DQError(st)
    return int(out.value)


def dq_paged_attention(q, q_dtype, q_stride, k_cache, v_cache, cache_dtype, k_scale, v_scale, page_table, lengths,
                       batch, q_heads, kv_heads, head_dim, num_pages, page_size, max_pages, window, sinks,
                       softmax_scale, out, lse, workspace, workspace_bytes, stream) -> int:
    """Raw call: pointers are ints (0/None for NULL). Returns the dq_status."""
    return _lib.dq_paged_attention(q, q_dtype, q_stride, k_cache, v_cache, cache_dtype, k_scale, v_scale, page_table,
                                   lengths, batch, q_heads, kv_heads, head_dim, num_pages, page_size, max_pages,
                                   window, sinks, softmax_scale, out, lse, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------- tensor-level helpers

def _torch():
    import torch

    return torch


_FLOAT_CODES: dict = {}


def _dtype_code(t) -> int:
    if not _FLOAT_CODES:
        torch = _torch()
        _FLOAT_CODES.update({torch.float32: DQ_F32, torch.float16: DQ_F16, torch.bfloat16: DQ_BF16})
    if t.dtype not in _FLOAT_CODES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _FLOAT_CODES[t.dtype]


def _dev_ptr(t, name: str) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_MODES = {"symmetric": DQ_SYMMETRIC, "asymmetric": DQ_ASYMMETRIC}
_YTYPES = {"int8": DQ_INT8, "int4": DQ_INT4X2, "int32": DQ_INT32}


def output_shapes(rows: int, cols: int, y_dtype: str):
    if y_dtype == "int8":
        return (rows, cols)
    if y_dtype == "int4":
        return (rows, cols // 2)
    return (rows, cols // 8)


def dynamic_quant(x, smooth=None, group_index=None, mode: str = "symmetric", y_dtype: str = "int8",
                  out=None, stream=None, check: bool = True):
    """Per-token dynamic quantization of CUDA tensor ``x`` (last dim = row).

    Returns ``(y, scale, offset, workspace)``: y int8 / uint8 (packed int4) /
    int32 (eight int4 per word) shaped like x with its last dim scaled;
    scale float32 (leading dims of x); offset float32 or None (symmetric);
    workspace (int32 tensor holding the status word) or None.
    ``out`` may pass preallocated ``(y, scale, offset, workspace)``.
    """
    torch = _torch()
    cols = int(x.shape[-1])
    rows = int(x.numel() // cols) if cols else 0
    lead = tuple(x.shape[:-1])
    m, yc = _MODES[mode], _YTYPES[y_dtype]
    ngroups = int(group_index.numel()) if group_index is not None else 0
    ws_bytes = dq_get_workspace_size(rows, cols, _dtype_code(x), m, yc, ngroups)
    if out is None:
        ydt = {"int8": torch.int8, "int4": torch.uint8, "int32": torch.int32}[y_dtype]
        y = torch.empty(lead + output_shapes(1, cols, y_dtype)[1:], dtype=ydt, device=x.device)
        scale = torch.empty(lead, dtype=torch.float32, device=x.device)
        offset = torch.empty(lead, dtype=torch.float32, device=x.device) if m == DQ_ASYMMETRIC else None
        ws = torch.empty((max(ws_bytes, 4) // 4,), dtype=torch.int32, device=x.device) if ws_bytes else None
    else:
        y, scale, offset, ws = out
    if stream is None:
        stream = _stream_of(x.get_device())
    st = dq_dynamic_quant(_dev_ptr(x, "x"), _dtype_code(x), rows, cols,
                          _dev_ptr(smooth, "smooth"), _dtype_code(smooth) if smooth is not None else DQ_F32,
                          _dev_ptr(group_index, "group_index"), ngroups, m, yc,
                          _dev_ptr(y, "y"), _dev_ptr(scale, "scale"), _dev_ptr(offset, "offset"),
                          _dev_ptr(ws, "workspace"), ws_bytes, stream)
    if check and st != DQ_OK:
        raise DQError(st)
    return y, scale, offset, ws


def ada_layernorm_quant(x, ada_scale, ada_shift, weight=None, bias=None, smooth=None, epsilon: float = 1e-6,
                        out=None, workspace=None, stream=None, check: bool = True):
    """Fused AdaLayerNorm + symmetric INT8 quantization of CUDA tensor ``x`` [batch, seq, hidden].

    Returns ``(out int8 [batch, seq, hidden], quant_scale float32 [batch, seq])``.
    ``workspace``: optional preallocated CUDA tensor of at least
    ``dq_ada_layernorm_quant_get_workspace_size`` bytes (16-byte aligned).
    """
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [batch, seq, hidden]")
    batch, seq, hidden = (int(d) for d in x.shape)
    pdt = _dtype_code(ada_scale)
    for name, p in (("ada_shift", ada_shift), ("weight", weight), ("bias", bias), ("smooth", smooth)):
        if p is not None and _dtype_code(p) != pdt:
            raise TypeError(f"{name} must have the dtype of ada_scale")
    ws_bytes = dq_ada_layernorm_quant_get_workspace_size(batch, seq, hidden, _dtype_code(x), pdt)
    if out is None:
        o = torch.empty((batch, seq, hidden), dtype=torch.int8, device=x.device)
        qs = torch.empty((batch, seq), dtype=torch.float32, device=x.device)
    else:
        o, qs = out
    if workspace is None and ws_bytes:
        workspace = torch.empty((ws_bytes + 15) // 16 * 4, dtype=torch.float32, device=x.device)
    if stream is None:
        stream = _stream_of(x.get_device())
    st = dq_ada_layernorm_quant(_dev_ptr(x, "x"), _dtype_code(x), batch, seq, hidden,
                                _dev_ptr(ada_scale, "ada_scale"), _dev_ptr(ada_shift, "ada_shift"),
                                _dev_ptr(weight, "weight"), _dev_ptr(bias, "bias"), _dev_ptr(smooth, "smooth"),
                                pdt, float(epsilon), _dev_ptr(o, "out"), _dev_ptr(qs, "quant_scale"),
                                _dev_ptr(workspace, "workspace"),
                                ws_bytes if workspace is not None else 0, stream)
    if check and st != DQ_OK:
        raise DQError(st)
    return o, qs


def dequant_per_token(y, scale, offset=None, y_dtype: str = "int8", cols: int | None = None,
                      out_dtype=None, out=None, stream=None, check: bool = True):
    """Per-token dequantization of CUDA codes ``y`` (AntiQuantize, PER_TOKEN).

    ``y``: int8 [rows, cols], uint8 [rows, cols/2] ("int4") or int32
    [rows, cols/8] ("int32"); ``scale`` / ``offset``: CUDA [rows] float
    tensors of one dtype; ``out_dtype``: torch.float32 / float16 / bfloat16
    (default: the scale's dtype). Returns the [rows, cols] output tensor.
    """
    torch = _torch()
    yc = _YTYPES[{"int8": "int8", "int4": "int4", "int32": "int32"}[y_dtype]]
    rows = int(y.shape[0]) if y.dim() else 0
    if cols is None:
        cols = int(y.shape[-1]) * {DQ_INT8: 1, DQ_INT4X2: 2, DQ_INT32: 8}[yc]
    sdt = _dtype_code(scale)
    if offset is not None and _dtype_code(offset) != sdt:
        raise TypeError("offset must have the dtype of scale")
    if out_dtype is None:
        out_dtype = scale.dtype
    if out is None:
        out = torch.empty((rows, cols), dtype=out_dtype, device=y.device)
    if stream is None:
        stream = _stream_of(y.get_device())
    st = dq_dequant_per_token(_dev_ptr(y, "y"), yc, rows, cols, _dev_ptr(scale, "scale"), _dev_ptr(offset, "offset"),
                              sdt, _dev_ptr(out, "out"), _dtype_code(out), stream)
    if check and st != DQ_OK:
        raise DQError(st)
    return out


def dequant_per_group(y, scale, offset=None, group_size: int = 32, k_dim: int = 1, y_dtype: str = "int8",
                      cols: int | None = None, out_dtype=None, out=None, stream=None, check: bool = True):
    """Per-group dequantization of CUDA codes ``y`` (AntiQuantize, PER_GROUP).

    ``scale`` / ``offset``: CUDA tables [rows, ceil(cols/g)] (``k_dim`` 1) or
    [ceil(rows/g), cols] (``k_dim`` 0) of one float dtype. Returns the
    [rows, cols] output tensor (``out_dtype`` defaults to the scale's dtype).
    """
    torch = _torch()
    yc = _YTYPES[y_dtype]
    rows = int(y.shape[0]) if y.dim() else 0
    if cols is None:
        cols = int(y.shape[-1]) * {DQ_INT8: 1, DQ_INT4X2: 2, DQ_INT32: 8}[yc]
    sdt = _dtype_code(scale)
    if offset is not None and _dtype_code(offset) != sdt:
        raise TypeError("offset must have the dtype of scale")
    if out is None:
        out = torch.empty((rows, cols), dtype=out_dtype or scale.dtype, device=y.device)
    if stream is None:
        stream = _stream_of(y.get_device())
    st = dq_dequant_per_group(_dev_ptr(y, "y"), yc, rows, cols, _dev_ptr(scale, "scale"), _dev_ptr(offset, "offset"),
                              sdt, int(group_size), int(k_dim), _dev_ptr(out, "out"), _dtype_code(out), stream)
    if check and st != DQ_OK:
        raise DQError(st)
    return out


def w8a8_gemm(a, b, a_scale, b_scale, out_dtype=None, out=None, accumulate: bool = False, stream=None,
              check: bool = True):
    """out = float(a @ b.T) * (a_scale[:, None] * b_scale[None, :]) (+ out).

    ``a``: CUDA int8 [M, K]; ``b``: CUDA int8 [N, K]; scales float32 [M], [N].
    Returns the [M, N] output (``out_dtype`` default float32).
    """
    torch = _torch()
    if a.dim() != 2 or b.dim() != 2 or a.dtype != torch.int8 or b.dtype != torch.int8:
        raise TypeError("a and b must be 2-D int8 tensors")
    m, k = (int(v) for v in a.shape)
    n = int(b.shape[0])
    if int(b.shape[1]) != k:
        raise ValueError(f"b must be [N, K] with the K of a ({k}), got {tuple(b.shape)}")
    for name, t, length in (("a_scale", a_scale, m), ("b_scale", b_scale, n)):
        if t.dtype != torch.float32 or t.numel() != length:
            raise TypeError(f"{name} must be float32 with {length} elements")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.float32, device=a.device)
    elif tuple(out.shape) != (m, n):
        raise ValueError(f"out must be [{m}, {n}], got {tuple(out.shape)}")
    if stream is None:
        stream = _stream_of(a.get_device())
    st = dq_w8a8_gemm(_dev_ptr(a, "a"), _dev_ptr(b, "b"), m, n, k, _dev_ptr(a_scale, "a_scale"),
                      _dev_ptr(b_scale, "b_scale"), _dev_ptr(out, "out"), _dtype_code(out), 1 if accumulate else 0,
                      stream)
    if check and st != DQ_OK:
        raise DQError(st)
    return out


# The helpers below check every tensor's shape, type, layout and device on the
# host: the kernels index by the sizes they are given. The launch goes to the
# tensors' device whatever the current one is, on that device's current stream
# or on `stream` (a cudaStream_t); what a helper allocates is allocated for that
# stream, so the allocator does not hand it on while the kernel still uses it.
# They are called once per layer and token, so each tensor is looked at in one
# call and the C entry point is called directly.

_ACTIVATIONS = {None: DQ_ACT_NONE, "none": DQ_ACT_NONE, "relu": DQ_ACT_RELU, "gelu": DQ_ACT_GELU,
                "gelu_tanh": DQ_ACT_GELU_TANH, "silu": DQ_ACT_SILU}


def _elsewhere(index: int, stream) -> bool:
    """Whether a call has to move to another device or stream than the current ones (see _on)."""
    return index >= 0 and (stream is not None or index != _torch().cuda.current_device())


def _on(index: int, stream):
    """The context that makes device `index` current, and `stream` when one is given."""
    torch = _torch()
    if stream is None:
        return torch.cuda.device(index)
    device = torch.device("cuda", index)
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream
                             else torch.cuda.default_stream(device))


def _stream_of(index: int) -> int:
    """The current stream of device `index`, without the Stream object around it where torch offers that.

    The last thing a helper asks before its launch: tensors on the CPU end here."""
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _arg(name: str, t, shape, dtype, index: int) -> int:
    """The pointer of a dense tensor after checking it."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(name: str, t, shape, dtype, index: int):
    """(pointer, elements between tokens) of [tokens, heads, head_dim] with dense heads, after checking it."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    row, head, one = t.stride()
    if one == 1 and head == shape[2] and row >= shape[1] * head:
        return t.data_ptr(), row
    return t.data_ptr(), _row_stride(name, t)


def _row_stride(name: str, t) -> int:
    tokens, heads, dim = t.shape
    row, head, one = t.stride()
    if t.numel() == 0 or tokens == 1:
        row = heads * dim
    elif row < heads * dim:
        raise ValueError(f"{name}: tokens overlap")
    if t.numel() and ((one != 1 and dim > 1) or (head != dim and heads > 1)):
        raise ValueError(f"{name}: the heads of a token must lie densely one after the other")
    return row


def w8a8_linear(a, b, a_scale, b_scale, bias=None, activation=None, residual=None, out_dtype=None, out=None,
                stream=None, check: bool = True):
    """out = act(float(a @ b.T) * (a_scale[:, None] * b_scale[None, :]) + bias) + residual.

    ``a``: CUDA int8 [M, K]; ``b``: CUDA int8 [N, K]; scales float32 [M], [N];
    ``bias``: float [N] or None; ``activation``: None / "none", "relu",
    "gelu", "gelu_tanh" or "silu"; ``residual``: [M, N] of the output's dtype
    or None, and may be ``out`` itself. Returns the [M, N] output
    (``out_dtype`` default: the residual's dtype, else float32).
    """
    torch = _torch()
    if a.dim() != 2 or b.dim() != 2 or a.dtype != torch.int8 or b.dtype != torch.int8:
        raise TypeError("a and b must be 2-D int8 tensors")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k:
        raise ValueError(f"b must be [N, K] with the K of a ({k}), got {tuple(b.shape)}")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else (torch.float32 if residual is None else residual.dtype)
    index = a.get_device()
    if _elsewhere(index, stream):
        with _on(index, stream):
            return w8a8_linear(a, b, a_scale, b_scale, bias, activation, residual, out_dtype, out, None, check)
    if out is None:
        out = a.new_empty((m, n), dtype=out_dtype)
    st = _lib.dq_w8a8_linear(
        _arg("a", a, (m, k), torch.int8, index), _arg("b", b, (n, k), torch.int8, index), m, n, k,
        _arg("a_scale", a_scale, (m,), torch.float32, index), _arg("b_scale", b_scale, (n,), torch.float32, index),
        None if bias is None else _arg("bias", bias, (n,), bias.dtype, index),
        DQ_F32 if bias is None else _dtype_code(bias), act,
        None if residual is None else _arg("residual", residual, (m, n), out_dtype, index),
        _arg("out", out, (m, n), out_dtype, index), _dtype_code(out), _stream_of(index))
    if check and st != DQ_OK:
        raise DQError(st)
    return out


def _weights(q_weight, k_weight, dim: int, index: int):
    """(q_weight pointer, k_weight pointer, dtype code)."""
    one = q_weight if q_weight is not None else k_weight
    if one is None:
        return None, None, DQ_F32
    return (None if q_weight is None else _arg("q_weight", q_weight, (dim,), one.dtype, index),
            None if k_weight is None else _arg("k_weight", k_weight, (dim,), one.dtype, index), _dtype_code(one))


def _norm_rope_shapes(q, k):
    """(q's shape, k's shape) of [tokens, heads, head_dim] tensors of the same tokens and head_dim."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    q_shape, k_shape = q.shape, k.shape
    if k_shape[0] != q_shape[0] or k_shape[2] != q_shape[2]:
        raise ValueError(f"k must be [{q_shape[0]}, kv_heads, {q_shape[2]}], got {list(k_shape)}")
    return q_shape, k_shape


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, epsilon: float = 1e-6,
                 interleaved: bool = False, out=None, stream=None, check: bool = True):
    """RMS norm of every query and key head with the position rotation, in one pass.

    ``q``, ``k``: CUDA float16 / bfloat16 [tokens, heads, head_dim], the heads
    of a token dense (slices of a fused projection work as they are);
    ``positions``: int32 [tokens]; ``inv_freq``: float32 [rope_dim / 2] or
    None (no rotation); weights: [head_dim] or None. ``out`` may pass
    ``(q_out, k_out)``, also ``(q, k)`` themselves. Returns ``(q_out, k_out)``.
    """
    torch = _torch()
    q_shape, k_shape = _norm_rope_shapes(q, k)
    (tokens, q_heads, dim), kv_heads = q_shape, k_shape[1]
    dtype, index, half = q.dtype, q.get_device(), 0 if inv_freq is None else inv_freq.numel()
    if _elsewhere(index, stream):
        with _on(index, stream):
            return qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, epsilon, interleaved, out, None, check)
    if out is None:
        q_out, k_out = q.new_empty(q_shape), q.new_empty(k_shape)
        outs = q_out.data_ptr(), q_heads * dim, k_out.data_ptr(), kv_heads * dim
    else:
        q_out, k_out = out
        outs = *_rows("q_out", q_out, q_shape, dtype, index), *_rows("k_out", k_out, k_shape, dtype, index)
    st = _lib.dq_qk_norm_rope(
        *_rows("q", q, q_shape, dtype, index), *_rows("k", k, k_shape, dtype, index), _dtype_code(q), tokens, q_heads,
        kv_heads, dim, *_weights(q_weight, k_weight, dim, index), epsilon,
        _arg("positions", positions, (tokens,), torch.int32, index),
        None if inv_freq is None else _arg("inv_freq", inv_freq, (half,), torch.float32, index), 2 * half,
        1 if interleaved else 0, *outs, _stream_of(index))
    if check and st != DQ_OK:
        raise DQError(st)
    return q_out, k_out


def _cache_args(k_cache, v_cache, k_scale, v_scale, kv_heads: int, dim: int, dtype, index: int):
    """(k pointer, v pointer, dtype code, k_scale pointer, v_scale pointer, num_pages, page_size) of a checked cache."""
    torch = _torch()
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, kv_heads, page_size, head_dim]")
    pages, page_size = k_cache.shape[0], k_cache.shape[2]
    shape = (pages, kv_heads, page_size, dim)
    if k_cache.dtype != torch.int8:
        return (_arg("k_cache", k_cache, shape, dtype, index), _arg("v_cache", v_cache, shape, dtype, index),
                _dtype_code(k_cache), None, None, pages, page_size)
    if k_scale is None or v_scale is None:
        raise ValueError("an int8 cache needs k_scale and v_scale")
    return (_arg("k_cache", k_cache, shape, torch.int8, index), _arg("v_cache", v_cache, shape, torch.int8, index),
            DQ_INT8, _arg("k_scale", k_scale, shape[:3], torch.float32, index),
            _arg("v_scale", v_scale, shape[:3], torch.float32, index), pages, page_size)


def qk_norm_rope_cache(q, k, v, positions, inv_freq, slots, k_cache, v_cache, k_scale=None, v_scale=None,
                       q_weight=None, k_weight=None, epsilon: float = 1e-6, interleaved: bool = False, out=None,
                       stream=None, check: bool = True):
    """``qk_norm_rope`` with the keys, and the values as they are, written into a paged cache.

    ``k_cache``, ``v_cache``: [num_pages, kv_heads, page_size, head_dim] of
    q's dtype, or int8 with float32 ``k_scale``, ``v_scale`` [num_pages,
    kv_heads, page_size]; ``slots``: int64 [tokens], page * page_size + row,
    negative for a token that is not stored. ``out`` may pass ``q_out``, also
    ``q`` itself. Returns ``q_out``; the caches are updated in place.
    """
    torch = _torch()
    q_shape, k_shape = _norm_rope_shapes(q, k)
    (tokens, q_heads, dim), kv_heads = q_shape, k_shape[1]
    dtype, index, half = q.dtype, q.get_device(), 0 if inv_freq is None else inv_freq.numel()
    if _elsewhere(index, stream):
        with _on(index, stream):
            return qk_norm_rope_cache(q, k, v, positions, inv_freq, slots, k_cache, v_cache, k_scale, v_scale,
                                      q_weight, k_weight, epsilon, interleaved, out, None, check)
    if out is None:
        out = q.new_empty(q_shape)
        outs = out.data_ptr(), q_heads * dim
    else:
        outs = _rows("out", out, q_shape, dtype, index)
    kc, vc, cdt, ks, vs, pages, page_size = _cache_args(k_cache, v_cache, k_scale, v_scale, kv_heads, dim, dtype, index)
    st = _lib.dq_qk_norm_rope_cache(
        *_rows("q", q, q_shape, dtype, index), *_rows("k", k, k_shape, dtype, index),
        *_rows("v", v, k_shape, dtype, index), _dtype_code(q), tokens, q_heads, kv_heads, dim,
        *_weights(q_weight, k_weight, dim, index), epsilon,
        _arg("positions", positions, (tokens,), torch.int32, index),
        None if inv_freq is None else _arg("inv_freq", inv_freq, (half,), torch.float32, index), 2 * half,
        1 if interleaved else 0, *outs, kc, vc, cdt, ks, vs,
        _arg("slots", slots, (tokens,), torch.int64, index), pages, page_size, _stream_of(index))
    if check and st != DQ_OK:
        raise DQError(st)
    return out


@functools.lru_cache(maxsize=None)
def _workspace_bytes(index: int, q_heads: int, kv_heads: int, dim: int, cache_dtype: int) -> int:
    """dq_paged_attention's workspace on device `index`, the current one; the batch does not matter."""
    return dq_paged_attention_get_workspace_size(1, q_heads, kv_heads, dim, cache_dtype)


def paged_attention(q, k_cache, v_cache, page_table, lengths, k_scale=None, v_scale=None, softmax_scale=None,
                    window: int = 0, sinks: int = 0, out=None, lse=None, workspace=None, stream=None,
                    check: bool = True):
    """Attention of one new token per sequence over a paged key-value cache.

    ``q``: CUDA float16 / bfloat16 [batch, q_heads, head_dim], dense heads;
    the cache as ``qk_norm_rope_cache`` writes it; ``page_table``: int32
    [batch, max_pages]; ``lengths``: int32 [batch], the new token included;
    ``softmax_scale``: default head_dim ** -0.5; ``window``: 0, or the number
    of last tokens that are visible beside the first ``sinks``; ``lse``: an
    optional float32 [batch, q_heads] output; ``workspace``: an optional
    preallocated CUDA tensor of at least
    ``dq_paged_attention_get_workspace_size`` bytes. Returns [batch, q_heads,
    head_dim] of q's dtype.
    """
    torch = _torch()
    if q.dim() != 3 or k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("q must be [batch, q_heads, head_dim], k_cache [num_pages, kv_heads, page_size, head_dim] "
                         "and page_table [batch, max_pages]")
    batch, q_heads, dim = shape = q.shape
    dtype, kv_heads, max_pages, index = q.dtype, k_cache.shape[1], page_table.shape[1], q.get_device()
    if _elsewhere(index, stream):
        with _on(index, stream):
            return paged_attention(q, k_cache, v_cache, page_table, lengths, k_scale, v_scale, softmax_scale, window,
                                   sinks, out, lse, workspace, None, check)
    if out is None:
        out = q.new_empty(shape)
        out_ptr = out.data_ptr()
    else:
        out_ptr = _arg("out", out, shape, dtype, index)
    kc, vc, cdt, ks, vs, pages, page_size = _cache_args(k_cache, v_cache, k_scale, v_scale, kv_heads, dim, dtype, index)
    if workspace is None:
        ws_bytes = _workspace_bytes(index, q_heads, kv_heads, dim, cdt)
        if ws_bytes:
            workspace = q.new_empty(ws_bytes, dtype=torch.uint8)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{index}")
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    ptr, stride = _rows("q", q, shape, dtype, index)
    st = _lib.dq_paged_attention(
        ptr, _dtype_code(q), stride, kc, vc, cdt, ks, vs,
        _arg("page_table", page_table, (batch, max_pages), torch.int32, index),
        _arg("lengths", lengths, (batch,), torch.int32, index), batch, q_heads, kv_heads, dim, pages, page_size,
        max_pages, window, sinks, dim ** -0.5 if softmax_scale is None else softmax_scale,
        out_ptr,
        None if lse is None else _arg("lse", lse, (batch, q_heads), torch.float32, index),
        None if workspace is None else workspace.data_ptr(), ws_bytes, _stream_of(index))
    if check and st != DQ_OK:
        raise DQError(st)
    return out
