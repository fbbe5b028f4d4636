"""Binding of the decode-path operators (include/sgemv_kv.h): the paged 4-bit KV cache and the
log-probabilities of the head's logits.

As in the package itself, each function carries the name of its C entry point and marshals arguments only:
tensors are checked for type, shape and strides, and their addresses passed on. Nothing here allocates
except the helpers `kv_cache`, `kv_workspace`, `kv_attention` and `logprobs`.
"""

from __future__ import annotations

import ctypes

import torch

from . import _check, _lib, _stream

SGEMV_F16 = 0
SGEMV_BF16 = 1
SGEMV_F32 = 2

KV_WORKSPACE = 32 << 20

EXPORTED_KV = ("sgemv_kv_layout_query", "sgemv_kv_plan", "sgemv_kv_append", "sgemv_kv_read", "sgemv_kv_attention",
               "sgemv_logprobs")

_DTYPE = {torch.float16: SGEMV_F16, torch.bfloat16: SGEMV_BF16, torch.float32: SGEMV_F32}


class KvLayout(ctypes.Structure):
    """sgemv_kv_layout: shape and byte layout of a paged 4-bit cache."""

    _fields_ = [(n, ctypes.c_int32) for n in ("heads", "dim", "group", "page", "n_pages", "reserved")] + \
        [(n, ctypes.c_uint64) for n in ("sub_bytes", "head_bytes", "page_bytes", "total_bytes")]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_ if name != "reserved"}

    def __repr__(self) -> str:
        return f"KvLayout({self.as_dict()})"


class KvQuery(ctypes.Structure):
    """sgemv_kv_query: what sgemv_kv_attention reads and writes beside the cache."""

    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "heads_q", "n_req", "n_tokens", "max_q", "window", "table_cols")] + \
        [("scale", ctypes.c_float)] + \
        [(n, ctypes.c_int64) for n in ("table_stride", "q_token_stride", "q_head_stride", "out_token_stride",
                                       "out_head_stride")] + \
        [(n, ctypes.c_void_p) for n in ("q_dev", "q_start_dev", "len_dev", "table_dev", "tree_dev", "out_dev", "lse_dev",
                                        "workspace_dev")] + \
        [("workspace_bytes", ctypes.c_uint64)]


_c, _p, _i, _l = ctypes, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
_lib.sgemv_kv_layout_query.argtypes = [_i] * 5 + [_c.POINTER(KvLayout)]
_lib.sgemv_kv_plan.argtypes = [_i, _i, _i, _p, _p, _p, _p, _i, _l] + [_p] * 7 + [_i, _p, _p]
_lib.sgemv_kv_append.argtypes = [_c.POINTER(KvLayout), _p, _i, _p, _l, _l, _p, _l, _l, _p, _i, _p, _p]
_lib.sgemv_kv_read.argtypes = [_c.POINTER(KvLayout), _p, _p, _i, _i, _p, _p, _p, _p]
_lib.sgemv_kv_attention.argtypes = [_c.POINTER(KvLayout), _p, _c.POINTER(KvQuery), _p, _p]
_lib.sgemv_logprobs.argtypes = [_p, _i, _i, _i, _l, _p, _i, _i] + [_p] * 8
for _name in EXPORTED_KV:
    getattr(_lib, _name).restype = ctypes.c_int


def _ptr(t):
    return None if t is None else t.data_ptr()


# The handle of a device's current stream without the Stream object that torch.cuda.current_stream() builds (2.9 us against 0.1).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
# The current device, which the library launches on, without torch.cuda's look at whether CUDA is up (a CUDA tensor is there).
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(t, what):
    """The device of t, where all tensors of its call have to be: the current one, since the library launches there."""
    try:
        dev = t.get_device()
    except AttributeError:
        raise TypeError(f"{what}: expected a torch.Tensor") from None
    if dev < 0:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if dev != _current():
        raise ValueError(f"{what}: on cuda:{dev}, but the current device is cuda:{_current()} (make it current around the call)")
    return dev


def _flat(t, dtype, numel, what, dev):
    """t is a contiguous tensor of dtype on the device, with numel elements (any number if None). (sgemv_kv_plan and
    sgemv_kv_attention, whose calls are short and have many tensors, ask the same in place first: a call here costs as much as
    the questions.)"""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and (numel is None or t.numel() == numel):
            return
    except AttributeError:
        raise TypeError(f"{what}: expected a torch.Tensor") from None
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor on cuda:{dev}")
    raise ValueError(f"{what}: expected {numel} elements, got {t.numel()}")


def _rows(t, shape, dtype, what, dev):
    """t is a tensor [tokens, heads, dim] of dtype on the device whose dims are contiguous: its token and head strides."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
            stride = t.stride()
            if stride[2] == 1:
                return stride
    except AttributeError:
        raise TypeError(f"{what}: expected a torch.Tensor") from None
    raise ValueError(f"{what}: expected a {dtype} tensor {tuple(shape)} on cuda:{dev} with contiguous dims")


def _cache_ok(layout, cache):
    """The device of the cache, which has the layout's bytes."""
    try:
        dev, size = cache.get_device(), cache.numel()
        if dev == _current() and cache.dtype is torch.uint8 and cache.is_contiguous() and size >= layout.total_bytes:
            return dev
    except AttributeError:
        raise TypeError("cache: expected a torch.Tensor") from None
    _flat(cache, torch.uint8, None, "cache", _device(cache, "cache"))
    raise ValueError(f"cache: need {layout.total_bytes} bytes")


def _table_ok(table, n_req, dev):
    """Columns and row stride of a block table."""
    if table.dtype is torch.int32 and table.get_device() == dev and table.dim() == 2:
        rows, cols = table.shape
        stride = table.stride()
        if rows == n_req and (rows == 0 or cols < 2 or stride[1] == 1) and (rows < 2 or stride[0] >= cols):
            return cols, max(stride[0], cols)
    raise ValueError(f"table: expected an int32 tensor [{n_req}, columns] on cuda:{dev} with contiguous rows")


def sgemv_kv_layout_query(heads: int, dim: int, group: int, page: int, n_pages: int) -> KvLayout:
    out = KvLayout()
    _check(_lib.sgemv_kv_layout_query(heads, dim, group, page, n_pages, ctypes.byref(out)), "sgemv_kv_layout_query")
    return out


def sgemv_kv_plan(length, keep, add, table, free, free_count, page: int, out, status=None, stream=None) -> None:
    """Block tables and slot maps of one step. length, keep (or None), add: int32 [n_req]; table: int32 [n_req, columns]
    and free: int32 [n_pages], both updated; free_count: int32 [1]. out = (length int32 [n_req], free_count int32 [1],
    q_start int32 [n_req + 1], slots int64 [n_slots], pos int32 [n_slots])."""
    o_length, o_count, o_start, o_slots, o_pos = out
    i32 = torch.int32
    try:
        dev = _device(length, "length")
        if length.dtype is not i32 or length.get_device() != dev or not length.is_contiguous():
            _flat(length, i32, None, "length", dev)
        n = length.numel()
        if keep is not None:
            if keep.dtype is not i32 or keep.get_device() != dev or not keep.is_contiguous() or keep.numel() != n:
                _flat(keep, i32, n, "keep", dev)
        if add.dtype is not i32 or add.get_device() != dev or not add.is_contiguous() or add.numel() != n:
            _flat(add, i32, n, "add", dev)
        cols, stride = _table_ok(table, n, dev)
        if free.dtype is not i32 or free.get_device() != dev or not free.is_contiguous():
            _flat(free, i32, None, "free", dev)
        if free_count.dtype is not i32 or free_count.get_device() != dev or not free_count.is_contiguous() or \
                free_count.numel() != 1:
            _flat(free_count, i32, 1, "free_count", dev)
        if o_length.dtype is not i32 or o_length.get_device() != dev or not o_length.is_contiguous() or o_length.numel() != n:
            _flat(o_length, i32, n, "out length", dev)
        if o_count.dtype is not i32 or o_count.get_device() != dev or not o_count.is_contiguous() or o_count.numel() != 1:
            _flat(o_count, i32, 1, "out free_count", dev)
        if o_start.dtype is not i32 or o_start.get_device() != dev or not o_start.is_contiguous() or o_start.numel() != n + 1:
            _flat(o_start, i32, n + 1, "out q_start", dev)
        if o_slots.dtype is not torch.int64 or o_slots.get_device() != dev or not o_slots.is_contiguous():
            _flat(o_slots, torch.int64, None, "out slots", dev)
        n_slots = o_slots.numel()
        if o_pos.dtype is not i32 or o_pos.get_device() != dev or not o_pos.is_contiguous() or o_pos.numel() != n_slots:
            _flat(o_pos, i32, n_slots, "out pos", dev)
        if status is not None:
            _flat(status, i32, None, "status", dev)
    except AttributeError:
        raise TypeError("sgemv_kv_plan: expected torch.Tensors") from None
    code = _lib.sgemv_kv_plan(n, page, free.numel(), length.data_ptr(), _ptr(keep), add.data_ptr(), table.data_ptr(), cols,
                              stride, free.data_ptr(), free_count.data_ptr(), o_length.data_ptr(), o_count.data_ptr(),
                              o_start.data_ptr(), o_slots.data_ptr(), o_pos.data_ptr(), n_slots, _ptr(status),
                              _raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_kv_plan")


def sgemv_kv_append(layout: KvLayout, cache, k, v, slots, status=None, stream=None) -> None:
    """Quantise k, v (fp16 or bf16 [tokens, heads, dim], any token and head strides) into the cache at slots (int64)."""
    dev = _cache_ok(layout, cache)
    _flat(slots, torch.int64, None, "slots", dev)
    n, dtype = slots.numel(), k.dtype
    shape = (n, layout.heads, layout.dim)
    ks, vs = _rows(k, shape, dtype, "k", dev), _rows(v, shape, dtype, "v", dev)
    if status is not None:
        _flat(status, torch.int32, None, "status", dev)
    code = _lib.sgemv_kv_append(ctypes.byref(layout), cache.data_ptr(), _DTYPE.get(dtype, -1), k.data_ptr(), ks[0], ks[1],
                                v.data_ptr(), vs[0], vs[1], slots.data_ptr(), n, _ptr(status),
                                _raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_kv_append")


def sgemv_kv_read(layout: KvLayout, cache, slots, k, v, status=None, stream=None) -> None:
    """The cached values of the tokens at slots into k, v (fp16, bf16 or fp32, contiguous [tokens, heads, dim])."""
    dev = _cache_ok(layout, cache)
    _flat(slots, torch.int64, None, "slots", dev)
    n, dtype = slots.numel(), k.dtype
    size = n * layout.heads * layout.dim
    _flat(k, dtype, size, "k", dev)
    _flat(v, dtype, size, "v", dev)
    if status is not None:
        _flat(status, torch.int32, None, "status", dev)
    code = _lib.sgemv_kv_read(ctypes.byref(layout), cache.data_ptr(), slots.data_ptr(), n, _DTYPE.get(dtype, -1),
                              k.data_ptr(), v.data_ptr(), _ptr(status), _raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_kv_read")


def sgemv_kv_attention(layout: KvLayout, cache, q, q_start, length, table, out, max_q: int, scale: float, workspace,
                       lse=None, window: int = 0, tree=None, status=None, stream=None) -> None:
    """Attention of the requests' new tokens over the cache. q, out: fp16 or bf16 [tokens, heads_q, dim] (any token and
    head strides); q_start int32 [n_req + 1]; length int32 [n_req], new tokens included; table int32 [n_req, columns];
    workspace: from kv_workspace(); lse: fp32 [tokens, heads_q] or None; tree: int64 [tokens] bit masks or None."""
    i32 = torch.int32
    try:
        dev = _cache_ok(layout, cache)
        n, heads, _ = shape = q.shape
        dtype = q.dtype
        if shape[2] != layout.dim:
            raise ValueError(f"q: expected rows of {layout.dim}")
        qs, os = _rows(q, shape, dtype, "q", dev), _rows(out, shape, dtype, "out", dev)
        if length.dtype is not i32 or length.get_device() != dev or not length.is_contiguous():
            _flat(length, i32, None, "length", dev)
        n_req = length.numel()
        if q_start.dtype is not i32 or q_start.get_device() != dev or not q_start.is_contiguous() or \
                q_start.numel() != n_req + 1:
            _flat(q_start, i32, n_req + 1, "q_start", dev)
        cols, stride = _table_ok(table, n_req, dev)
        if workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
            _flat(workspace, torch.uint8, None, "workspace", dev)
        if lse is not None:
            _flat(lse, torch.float32, n * heads, "lse", dev)
        if tree is not None:
            _flat(tree, torch.int64, n, "tree", dev)
        if status is not None:
            _flat(status, i32, None, "status", dev)
    except AttributeError:
        raise TypeError("sgemv_kv_attention: expected torch.Tensors") from None
    args = KvQuery(_DTYPE.get(dtype, -1), heads, n_req, n, max_q, window, cols, scale, stride, qs[0], qs[1], os[0], os[1],
                   q.data_ptr(), q_start.data_ptr(), length.data_ptr(), table.data_ptr(), _ptr(tree), out.data_ptr(),
                   _ptr(lse), workspace.data_ptr(), workspace.numel())
    code = _lib.sgemv_kv_attention(ctypes.byref(layout), cache.data_ptr(), ctypes.byref(args), _ptr(status),
                                   _raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_kv_attention")


def sgemv_logprobs(logits, out, tokens=None, status=None, stream=None) -> None:
    """Log-probabilities of logits (fp16, bf16 or fp32 [rows, vocab], contiguous vocabulary). tokens: int32 [rows, n] or
    None. out = (tok_logp fp32 [rows, n], lse fp32 [rows], entropy fp32 [rows], top_tok int32 [rows, top],
    top_logp fp32 [rows, top], logp fp32 [rows, vocab]), any of them None; top is top_tok's width."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits: expected a torch.Tensor")
    dev = _device(logits, "logits")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits: expected a CUDA tensor [rows, vocab] with a contiguous vocabulary")
    rows, vocab = logits.shape
    stride = vocab if rows < 2 else logits.stride(0)
    if stride < vocab:
        raise ValueError("logits: rows overlap (a row stride below the vocabulary)")
    tok_logp, lse, entropy, top_tok, top_logp, logp = out
    f32, n_tok, top = torch.float32, 0, 0
    if (tokens is None) != (tok_logp is None) or (top_tok is None) != (top_logp is None):
        raise ValueError("tokens and out tok_logp, and out top_tok and top_logp, come together")
    if tokens is not None:
        n_tok = tokens.shape[1] if tokens.dim() == 2 else 1
        _flat(tokens, torch.int32, rows * n_tok, "tokens", dev)
        _flat(tok_logp, f32, rows * n_tok, "out tok_logp", dev)
    if top_tok is not None:
        top = top_tok.shape[1]
        _flat(top_tok, torch.int32, rows * top, "out top_tok", dev)
        _flat(top_logp, f32, rows * top, "out top_logp", dev)
    for t, n, what in ((lse, rows, "out lse"), (entropy, rows, "out entropy"), (logp, rows * vocab, "out logp")):
        if t is not None:
            _flat(t, f32, n, what, dev)
    if status is not None:
        _flat(status, torch.int32, None, "status", dev)
    code = _lib.sgemv_logprobs(logits.data_ptr(), _DTYPE.get(logits.dtype, -1), rows, vocab, stride, _ptr(tokens), n_tok, top,
                               _ptr(tok_logp), _ptr(lse), _ptr(entropy), _ptr(top_tok), _ptr(top_logp), _ptr(logp), _ptr(status),
                               _raw_stream(dev) if stream is None else _stream(stream))
    if code:
        _check(code, "sgemv_logprobs")


# ---------------------------------------------------------------------------------------------- helpers

def kv_cache(layout: KvLayout, device="cuda"):
    """The bytes of a cache of this layout (uninitialised: what was never written is never used)."""
    return torch.empty(layout.total_bytes, dtype=torch.uint8, device=device)


def kv_workspace(device="cuda"):
    """Workspace of sgemv_kv_attention, zeroed as its first call needs it; one for each stream that calls it."""
    return torch.zeros(KV_WORKSPACE, dtype=torch.uint8, device=device)


def kv_attention(layout: KvLayout, cache, q, q_start, length, table, max_q: int, scale: float, workspace, window: int = 0,
                 tree=None, status=None, stream=None, lse=None):
    """sgemv_kv_attention into a new contiguous tensor, which it returns; lse: fp32 [tokens, heads_q] to write, or None."""
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    sgemv_kv_attention(layout, cache, q, q_start, length, table, out, max_q, scale, workspace, lse, window, tree, status,
                       stream)
    return out


def logprobs(logits, tokens=None, top: int = 0, full: bool = False, status=None, stream=None) -> dict:
    """sgemv_logprobs into new tensors: {"lse", "entropy"} and, where asked for, {"tok_logp", "top_tok", "top_logp",
    "logp"}."""
    rows, vocab = logits.shape
    f = dict(dtype=torch.float32, device=logits.device)
    got = {"lse": torch.empty(rows, **f), "entropy": torch.empty(rows, **f)}
    if tokens is not None:
        got["tok_logp"] = torch.empty(tokens.shape, **f)
    if top:
        got["top_tok"] = torch.empty((rows, top), dtype=torch.int32, device=logits.device)
        got["top_logp"] = torch.empty((rows, top), **f)
    if full:
        got["logp"] = torch.empty((rows, vocab), **f)
    sgemv_logprobs(logits, tuple(got.get(n) for n in ("tok_logp", "lse", "entropy", "top_tok", "top_logp", "logp")),
                   tokens, status, stream)
    return got
