"""Binding of the prompt-path operators (include/sgemv_prompt.h): matrices in block-scaled 4-bit floating point and their product, and
causal attention over packed prompts.

As in the package itself, each function carries the name of its C entry point and marshals arguments only: tensors are checked for type,
shape and strides, and their addresses passed on. Nothing here allocates except the helpers `fp4_quantize`, `fp4_product` and
`prompt_attention`.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import _allocate, _check, _lib, _stream
from . import kv as _kv
from .kv import _DTYPE, _device, _flat, _rows

EXPORTED_PROMPT = ("sgemv_fp4_layout_query", "sgemv_fp4_quantize", "sgemv_fp4_read", "sgemv_fp4_product", "sgemv_prompt_attention")


class Fp4Layout(ctypes.Structure):
    """sgemv_fp4_layout: shape and byte layout of a matrix in block-scaled 4-bit floating point."""

    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "k", "block", "tile", "kp", "reserved")] + \
        [(n, ctypes.c_uint64) for n in ("scale_off", "row_off", "total_bytes")]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_ if name != "reserved"}

    def __repr__(self) -> str:
        return f"Fp4Layout({self.as_dict()})"


class PromptQuery(ctypes.Structure):
    """sgemv_prompt_query: what sgemv_prompt_attention reads and writes."""

    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "heads_q", "heads", "dim", "n_req", "n_tokens", "causal", "window")] + \
        [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)] + \
        [(n, ctypes.c_int64) for n in ("q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride", "v_token_stride",
                                       "v_head_stride", "out_token_stride", "out_head_stride")] + \
        [(n, ctypes.c_void_p) for n in ("q_dev", "k_dev", "v_dev", "start_dev", "length_dev", "out_dev", "lse_dev")]


_U8 = torch.uint8
# PromptQuery's bytes: filling them in at once takes 0.6 us, a Structure field by field 2.
_QUERY = struct.Struct("=8ifi8q7Q")
assert _QUERY.size == ctypes.sizeof(PromptQuery)

_c, _p, _i, _l = ctypes, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
_lib.sgemv_fp4_layout_query.argtypes = [_i] * 3 + [_c.POINTER(Fp4Layout)]
_lib.sgemv_fp4_quantize.argtypes = [_c.POINTER(Fp4Layout), _p, _i, _l, _p, _p, _p]
_lib.sgemv_fp4_read.argtypes = [_c.POINTER(Fp4Layout), _p, _p, _i, _l, _p]
_lib.sgemv_fp4_product.argtypes = [_c.POINTER(Fp4Layout), _p, _c.POINTER(Fp4Layout), _p, _p, _i, _l, _p, _p]
_lib.sgemv_prompt_attention.argtypes = [_p, _p, _p]
for _name in EXPORTED_PROMPT:
    getattr(_lib, _name).restype = ctypes.c_int


def _row_stride(t, rows, cols, what, dev):
    """t is a tensor [rows, cols] on the device with contiguous columns: its row stride."""
    try:
        if t.get_device() == dev and t.shape == (rows, cols):
            s0, s1 = t.stride()
            if (s1 == 1 or cols < 2) and (s0 >= cols or rows < 2):
                return s0 if rows > 1 else cols
    except AttributeError:
        raise TypeError(f"{what}: expected a torch.Tensor") from None
    raise ValueError(f"{what}: expected a tensor [{rows}, {cols}] on cuda:{dev} with contiguous columns and rows that do not overlap")


def _packed(layout, t, what):
    """The device of the bytes of a 4-bit matrix."""
    try:
        dev, size = t.get_device(), t.numel()
        if dev == _kv._current() and t.dtype is torch.uint8 and t.is_contiguous() and size >= layout.total_bytes:
            return dev
    except AttributeError:
        raise TypeError(f"{what}: expected a torch.Tensor") from None
    _flat(t, torch.uint8, None, what, _device(t, what))
    raise ValueError(f"{what}: need {layout.total_bytes} bytes")


def sgemv_fp4_layout_query(rows: int, k: int, block: int) -> Fp4Layout:
    out = Fp4Layout()
    _check(_lib.sgemv_fp4_layout_query(rows, k, block, ctypes.byref(out)), "sgemv_fp4_layout_query")
    return out


def sgemv_fp4_quantize(layout: Fp4Layout, packed, x, status=None, stream=None) -> None:
    """The 4-bit matrix of x (fp16 or bf16 [rows, k], any row stride) into packed (uint8, layout.total_bytes)."""
    # (the usual case asked in place, as in sgemv_kv_plan: a call here costs as much as the questions)
    try:
        dev, shape, stride = packed.get_device(), x.shape, x.stride()
        usual = packed.dtype is _U8 and packed.numel() >= layout.total_bytes and packed.is_contiguous() and x.get_device() == dev and \
            dev == _kv._current() and shape == (layout.rows, layout.k) and stride[1] == 1 and stride[0] >= shape[1]
    except (AttributeError, IndexError):
        usual = False
    if usual:
        row = stride[0]
    else:
        dev = _packed(layout, packed, "packed")
        row = _row_stride(x, layout.rows, layout.k, "x", dev)
    if status is not None:
        _flat(status, torch.int32, None, "status", dev)
    code = _lib.sgemv_fp4_quantize(ctypes.byref(layout), x.data_ptr(), _DTYPE.get(x.dtype, -1), row, packed.data_ptr(),
                                   None if status is None else status.data_ptr(),
                                   _kv._raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_fp4_quantize")


def sgemv_fp4_read(layout: Fp4Layout, packed, out, stream=None) -> None:
    """The values that a 4-bit matrix stands for into out (fp16, bf16 or fp32 [rows, k], any row stride)."""
    dev = _packed(layout, packed, "packed")
    stride = _row_stride(out, layout.rows, layout.k, "out", dev)
    code = _lib.sgemv_fp4_read(ctypes.byref(layout), packed.data_ptr(), out.data_ptr(), _DTYPE.get(out.dtype, -1), stride,
                               _kv._raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_fp4_read")


def sgemv_fp4_product(w_layout: Fp4Layout, w, x_layout: Fp4Layout, x, y, status=None, stream=None) -> None:
    """y[t][n] = sum over k of x[t][k] w[n][k] of two 4-bit matrices; y: fp16 or bf16 [x rows, w rows], any row stride."""
    try:
        dev, shape, stride = w.get_device(), y.shape, y.stride()
        usual = w.dtype is _U8 and x.dtype is _U8 and w.numel() >= w_layout.total_bytes and x.numel() >= x_layout.total_bytes and \
            w.is_contiguous() and x.is_contiguous() and x.get_device() == dev and y.get_device() == dev and dev == _kv._current() and \
            shape == (x_layout.rows, w_layout.rows) and stride[1] == 1 and stride[0] >= shape[1]
    except (AttributeError, IndexError):
        usual = False
    if usual:
        row = stride[0]
    else:
        dev = _packed(w_layout, w, "w")
        _packed(x_layout, x, "x")
        row = _row_stride(y, x_layout.rows, w_layout.rows, "y", dev)
    if status is not None:
        _flat(status, torch.int32, None, "status", dev)
    code = _lib.sgemv_fp4_product(ctypes.byref(w_layout), w.data_ptr(), ctypes.byref(x_layout), x.data_ptr(), y.data_ptr(),
                                  _DTYPE.get(y.dtype, -1), row, None if status is None else status.data_ptr(),
                                  _kv._raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_fp4_product")


def sgemv_prompt_attention(q, k, v, start, out, scale: float, length=None, lse=None, causal: bool = True, window: int = 0, status=None,
                           stream=None) -> None:
    """Attention of each request's tokens over its own keys and values. q, out: fp16 or bf16 [tokens, heads_q, dim], k, v: the same type
    [tokens, heads, dim] (any token and head strides); start: int32 [n_req + 1]; length: int32 [n_req] or None (requests padded at their
    ends); lse: fp32 [tokens, heads_q] or None."""
    i32 = torch.int32
    try:
        dev, dtype, shape = q.get_device(), q.dtype, q.shape
        if dev < 0 or dev != _kv._current():
            _device(q, "q")
        n, heads_q, dim = shape
        kv_shape = k.shape
        # (asked in one go: a call for each tensor costs as much as the questions)
        if not (k.dtype is dtype and v.dtype is dtype and out.dtype is dtype and k.get_device() == dev and v.get_device() == dev and
                out.get_device() == dev and out.shape == shape and v.shape == kv_shape and len(kv_shape) == 3 and kv_shape[0] == n and
                kv_shape[2] == dim):
            if k.dim() != 3:
                raise ValueError("k: expected a tensor [tokens, heads, dim]")
            _rows(out, shape, dtype, "out", dev)
            kv_shape = (n, k.shape[1], dim)
            _rows(k, kv_shape, dtype, "k", dev)
            _rows(v, kv_shape, dtype, "v", dev)
        q0, q1, q2 = q.stride()
        k0, k1, k2 = k.stride()
        v0, v1, v2 = v.stride()
        o0, o1, o2 = out.stride()
        if not q2 == k2 == v2 == o2 == 1:
            raise ValueError("q, k, v, out: expected contiguous dims")
        if start.dtype is not i32 or start.get_device() != dev or not start.is_contiguous():
            _flat(start, i32, None, "start", dev)
        n_req = start.numel() - 1
        if length is not None:
            _flat(length, i32, n_req, "length", dev)
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous() or lse.numel() != n * heads_q:
                _flat(lse, torch.float32, n * heads_q, "lse", dev)
        if status is not None:
            _flat(status, i32, None, "status", dev)
    except AttributeError:
        raise TypeError("sgemv_prompt_attention: expected torch.Tensors") from None
    try:
        query = _QUERY.pack(_DTYPE.get(dtype, -1), heads_q, kv_shape[1], dim, n_req, n, 1 if causal else 0, window, scale, 0, q0, q1, k0, k1, v0, v1,
                            o0, o1, q.data_ptr(), k.data_ptr(), v.data_ptr(), start.data_ptr(), 0 if length is None else length.data_ptr(),
                            out.data_ptr(), 0 if lse is None else lse.data_ptr())
    except (struct.error, OverflowError) as e:  # (a scale that is no binary32 is the latter)
        raise ValueError(f"sgemv_prompt_attention: {e}") from None
    code = _lib.sgemv_prompt_attention(query, None if status is None else status.data_ptr(),
                                       _kv._raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_prompt_attention")


# ---------------------------------------------------------------------------------------------- helpers

def fp4_quantize(x, block: int = 16, status=None, stream=None):
    """(layout, bytes) of the 4-bit matrix of x (fp16 or bf16 [rows, k])."""
    layout = sgemv_fp4_layout_query(x.shape[0], x.shape[1], block)
    packed = _allocate(stream, lambda: torch.empty(layout.total_bytes, dtype=torch.uint8, device=x.device))
    sgemv_fp4_quantize(layout, packed, x, status, stream)
    return layout, packed


def fp4_product(w_layout: Fp4Layout, w, x_layout: Fp4Layout, x, dtype=torch.bfloat16, status=None, stream=None):
    """sgemv_fp4_product into a new contiguous tensor [x rows, w rows] of dtype, which it returns."""
    y = _allocate(stream, lambda: torch.empty((x_layout.rows, w_layout.rows), dtype=dtype, device=w.device))
    sgemv_fp4_product(w_layout, w, x_layout, x, y, status, stream)
    return y


def prompt_attention(q, k, v, start, scale: float, length=None, lse=None, causal: bool = True, window: int = 0, status=None, stream=None):
    """sgemv_prompt_attention into a new contiguous tensor, which it returns (rows of no request hold anything)."""
    out = _allocate(stream, lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device))
    sgemv_prompt_attention(q, k, v, start, out, scale, length, lse, causal, window, status, stream)
    return out
