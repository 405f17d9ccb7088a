"""Paged K/V cache in NVFP4: planning, quantizing writes and attention.

Binding of the ``nvfp4_kv_*`` entry points (``include/nvfp4rq.h``), which say
what each computes and how a record is laid out.  A step of a server:

    plan = kv_plan(cached, added, table, free, head, page_size, tokens)
    kv_append(k, v, plan.slots, cache, amax)
    out = kv_attention(q, cache, amax, table, plan.cu_q, plan.kv_lens, max_q=most)

with ``most`` the most tokens that any request of the step adds.
``cache`` is a uint8 tensor [pages, kv_heads, page bytes] (kv_cache makes
one); its page size follows from the head dimension of k or q.  ``amax`` holds
the maxima of rotated K and V that fix the two global scales, for instance
from ``rotamax`` on a calibration tensor.

A call runs on PyTorch's current stream, or on ``stream``; what it allocates is
memory of that stream, and waiting for it before using the outputs elsewhere
is the caller's part.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import _buf, _check, _empty, _p, _ptr, lib

__all__ = ["KvPlan", "kv_append", "kv_attention", "kv_attention_workspace", "kv_cache", "kv_page_bytes", "kv_plan"]

_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_int = ctypes.c_int
_strides2 = _i64 * 2


class _Cache(ctypes.Structure):
    _fields_ = [("data", _p), ("amax", _p), ("pages", _i64), ("kv_heads", _i32), ("head_dim", _i32),
                ("page_size", _i32), ("rotate", _i32)]


class _Batch(ctypes.Structure):
    _fields_ = [("table", _p), ("table_width", _i64), ("cu_q", _p), ("kv_lens", _p), ("requests", _i64),
                ("max_q", _i64), ("max_kv", _i64), ("causal", _i32), ("window", _i32), ("scale", ctypes.c_float)]


_SIGS = {
    "nvfp4_kv_plan": [_p, _p, _i64, _i32, _p, _i64, _p, _i64, _p, _p, _i64, _p, _p, _p, _p, _p],
    "nvfp4_kv_append": [_p, _p, _i64, _p, _p, _p, _p, _p],
    "nvfp4_kv_append_f32": [_p, _p, _i64, _p, _p, _p, _p, _p],
    "nvfp4_kv_attention": [_p, _i64, _i32, _p, _p, _p, _p, _p, _p, _i64, _p],
    "nvfp4_kv_attention_f32": [_p, _i64, _i32, _p, _p, _p, _p, _p, _p, _i64, _p],
}
for _name, _args in _SIGS.items():
    getattr(lib, _name).argtypes = _args
    getattr(lib, _name).restype = _int
lib.nvfp4_kv_page_bytes.argtypes = [_i32, _i32]
lib.nvfp4_kv_page_bytes.restype = _i64
lib.nvfp4_kv_attention_workspace.argtypes = [_i64, _i32, _p, _p]
lib.nvfp4_kv_attention_workspace.restype = _i64


def _within(value: int, most: int, name: str) -> int:
    """value, 0 .. most; a larger one would lose its high bits on the way."""
    if not 0 <= value <= most:
        raise ValueError(f"{name} must be from 0 to {most}, got {value}")
    return value


_MOST32, _MOST64 = (1 << 31) - 1, (1 << 63) - 1


def kv_page_bytes(page_size: int, head_dim: int) -> int:
    """Bytes that a page takes for one head, K and V together."""
    _within(page_size, _MOST32, "page_size")
    _within(head_dim, _MOST32, "head_dim")
    n = int(lib.nvfp4_kv_page_bytes(page_size, head_dim))
    if n < 0:
        raise ValueError(f"no page layout for page_size {page_size} and head_dim {head_dim}: page_size is a power "
                         "of two from 16 to 65536, head_dim 64, 128 or 256")
    return n


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int, device="cuda") -> torch.Tensor:
    """An empty (zeroed) cache: uint8 [pages, kv_heads, kv_page_bytes]."""
    return torch.zeros(pages, kv_heads, kv_page_bytes(page_size, head_dim), dtype=torch.uint8, device=device)


def _page_size(cache: torch.Tensor, head_dim: int) -> int:
    size, rest = divmod(cache.shape[2] * 8, 9 * head_dim)
    if rest or size < 16 or size > 65536 or size & (size - 1):
        raise ValueError(f"cache pages of {cache.shape[2]} bytes a head hold no power of two (16 to 65536) of tokens "
                         f"of head_dim {head_dim}")
    return size


def _cache_arg(cache, amax, heads: int, head_dim: int, rotate: bool, device: torch.device) -> _Cache:
    if not isinstance(cache, torch.Tensor):
        raise TypeError("cache must be a tensor")
    if cache.dim() != 3:
        raise ValueError("cache must be 3-D [pages, kv_heads, page bytes]")
    _buf(cache, 0, torch.uint8, device, "cache")
    _buf(amax, 2, torch.float32, device, "amax")
    if head_dim not in (64, 128, 256):
        raise ValueError(f"head_dim must be 64, 128 or 256, got {head_dim}")
    if heads % max(1, cache.shape[1]):
        raise ValueError(f"{heads} heads do not divide into the cache's {cache.shape[1]}")
    return _Cache(_ptr(cache), _ptr(amax), cache.shape[0], cache.shape[1], head_dim, _page_size(cache, head_dim),
                  int(bool(rotate)))


def _rows(t, name: str, dtype=None, device=None):
    """A [tokens, heads, head_dim] operand and its two strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != (dtype or t.dtype) or t.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"{name} must be {dtype or 'bfloat16 or float32'}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, head_dim]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the first argument on {device}")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be contiguous along head_dim")
    shape, size = t.shape, t.element_size()
    ts, hs = t.stride()[:2]
    if shape[0] <= 1:
        ts = 0
    if shape[1] <= 1:
        hs = 0
    if ts * size % 16 or hs * size % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}'s rows must start at multiples of 16 bytes")
    return _strides2(ts, hs)


def _on_device(fn):
    """Run the call with its first tensor's GPU as the current device; changing
    to it and back only where it is another one (1.5 us)."""
    first = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, **kwargs):
        t = args[0] if args else kwargs.get(first)
        if isinstance(t, torch.Tensor) and t.is_cuda and t.device.index != torch.cuda.current_device():
            with torch.cuda.device(t.device):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return call


def _stream(device: torch.device, stream) -> int:
    """The stream's handle; PyTorch's current one without the object around it
    (2 us) when None."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


class KvPlan(NamedTuple):
    """What kv_plan computes, on the device."""
    slots: torch.Tensor    # int64 [tokens]: where each new token goes, -1 for none
    cu_q: torch.Tensor     # int32 [requests + 1]: first row of each request's new tokens
    kv_lens: torch.Tensor  # int32 [requests]: cached + added
    head: torch.Tensor     # int32 [1]: entries of the free list taken so far
    missing: torch.Tensor  # int32 [2]: pages and slots that there was no room for


@_on_device
def kv_plan(cached: torch.Tensor, added: torch.Tensor, table: torch.Tensor, free: torch.Tensor, head: torch.Tensor,
            page_size: int, tokens: int, out: KvPlan | None = None, stream=None) -> KvPlan:
    """One step's bookkeeping.  cached, added: int32 [requests] tokens that each
    request has and adds; table: int32 [requests, width], whose new entries are
    written; free: int32 list of free pages, taken from head (int32 [1]) on;
    tokens: rows of the step, at least the sum of added (the rest get slot -1)."""
    if not isinstance(cached, torch.Tensor) or not isinstance(table, torch.Tensor):
        raise TypeError("cached and table must be tensors")
    if not cached.is_cuda:
        raise ValueError("cached must be a device tensor")
    device, n = cached.device, cached.numel()
    _buf(cached, n, torch.int32, device, "cached")
    _buf(added, n, torch.int32, device, "added")
    if table.dim() != 2 or table.shape[0] != n:
        raise ValueError("table must be 2-D [requests, width]")
    _buf(table, 0, torch.int32, device, "table")
    _buf(free, 0, torch.int32, device, "free")
    _buf(head, 1, torch.int32, device, "head")
    _within(page_size, _MOST32, "page_size")
    _within(tokens, _MOST32, "tokens")
    if out is None:
        ints = _empty(2 * n + 4, torch.int32, device, stream).split((n + 1, n, 1, 2))
        out = KvPlan(_empty(tokens, torch.int64, device, stream), *ints)
    else:
        _buf(out[0], tokens, torch.int64, device, "slots")
        for t, size, name in zip(out[1:], (n + 1, n, 1, 2), KvPlan._fields[1:]):
            _buf(t, size, torch.int32, device, name)
    _check("nvfp4_kv_plan", lib.nvfp4_kv_plan(
        _ptr(cached), _ptr(added), n, page_size, _ptr(table), table.shape[1], _ptr(free), free.numel(), _ptr(head),
        _ptr(out[0]), tokens, _ptr(out[1]), _ptr(out[2]), _ptr(out[3]), _ptr(out[4]), _stream(device, stream)))
    return out


@_on_device
def kv_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, amax: torch.Tensor,
              rotate: bool = True, stream=None) -> torch.Tensor:
    """Rotates, quantizes and writes k and v (bfloat16 or float32 [tokens,
    kv_heads, head_dim], rows of 16-byte aligned strides) to slots (int64
    [tokens]; -1 skips a row) of the cache, which it returns."""
    ks = _rows(k, "k")
    vs = _rows(v, "v", k.dtype, k.device)
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    c = _cache_arg(cache, amax, k.shape[1], k.shape[2], rotate, k.device)
    if k.shape[1] != c.kv_heads:
        raise ValueError(f"k has {k.shape[1]} heads, the cache {c.kv_heads}")
    _buf(slots, k.shape[0], torch.int64, k.device, "slots")
    fn = "nvfp4_kv_append" if k.dtype == torch.bfloat16 else "nvfp4_kv_append_f32"
    _check(fn, getattr(lib, fn)(_ptr(k), _ptr(v), k.shape[0], ks, vs, _ptr(slots), ctypes.byref(c),
                                _stream(k.device, stream)))
    return cache


class _NoGradient(torch.autograd.Function):
    """The result of a call on x that has no backward pass, kept in x's graph so
    that one through it is refused rather than lost."""

    @staticmethod
    def forward(ctx, x, call):
        return call()

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("kv_attention has no backward pass: call it on q.detach() or under torch.no_grad()")


def _batch_arg(q, cache, amax, table, cu_q, kv_lens, max_q, max_kv, causal, window, scale, rotate):
    device = q.device
    c = _cache_arg(cache, amax, _within(q.shape[1], _MOST32, "q's heads"), q.shape[2], rotate, device)
    if not isinstance(table, torch.Tensor):
        raise TypeError("table must be a tensor")
    if table.dim() != 2:
        raise ValueError("table must be 2-D [requests, width]")
    n, width = table.shape
    _buf(table, 0, torch.int32, device, "table")
    _buf(cu_q, n + 1, torch.int32, device, "cu_q")
    _buf(kv_lens, n, torch.int32, device, "kv_lens")
    max_q = q.shape[0] if max_q is None else _within(max_q, _MOST64, "max_q")
    max_kv = width * c.page_size if max_kv is None else _within(max_kv, _MOST64, "max_kv")
    b = _Batch(_ptr(table), width, _ptr(cu_q), _ptr(kv_lens), n, max_q, max_kv, int(bool(causal)),
               _within(window, _MOST32, "window"), q.shape[2] ** -0.5 if scale is None else scale)
    return c, b


@_on_device
def kv_attention_workspace(q: torch.Tensor, cache: torch.Tensor, amax: torch.Tensor, table: torch.Tensor,
                           cu_q: torch.Tensor, kv_lens: torch.Tensor, max_q: int | None = None,
                           max_kv: int | None = None, causal: bool = True, window: int = 0,
                           scale: float | None = None, rotate: bool = True) -> int:
    """Bytes of workspace that kv_attention takes for these arguments."""
    _rows(q, "q")
    c, b = _batch_arg(q, cache, amax, table, cu_q, kv_lens, max_q, max_kv, causal, window, scale, rotate)
    n = int(lib.nvfp4_kv_attention_workspace(q.shape[0], q.shape[1], ctypes.byref(c), ctypes.byref(b)))
    if n < 0:
        raise ValueError("no launch for these shapes")
    return n


@_on_device
def kv_attention(q: torch.Tensor, cache: torch.Tensor, amax: torch.Tensor, table: torch.Tensor, cu_q: torch.Tensor,
                 kv_lens: torch.Tensor, max_q: int | None = None, max_kv: int | None = None, causal: bool = True,
                 window: int = 0, scale: float | None = None, rotate: bool = True, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the new tokens over their requests' pages.  q: bfloat16 or
    float32 [tokens, q_heads, head_dim]; request r's rows are cu_q[r] ..
    cu_q[r + 1] - 1 and its keys the first kv_lens[r] tokens of table[r], its new
    ones included.  max_q and max_kv: the most of either that any request has
    (bounds from the shapes when None: all tokens, the table's width); they shape
    the launch, not the result.  Give max_q where single tokens of many requests
    come together: 64 of them over 8192 keys take 80 us with it and 110 without.
    scale: head_dim ** -0.5 when None.  Rows in no request are left as they were
    in out, and hold anything, NaN included, where out is None.  workspace: a
    uint8 tensor of kv_attention_workspace bytes, allocated when None; calls that
    share one must be ordered.  No gradients: a backward pass that reaches the
    result raises, unless it was written to the caller's out, which keeps no
    record of q."""
    if out is None and torch.is_grad_enabled() and isinstance(q, torch.Tensor) and q.requires_grad:
        return _NoGradient.apply(q, lambda: kv_attention(
            q.detach(), cache, amax, table, cu_q, kv_lens, max_q, max_kv, causal, window, scale, rotate, None,
            workspace, stream))
    qs = _rows(q, "q")
    c, b = _batch_arg(q, cache, amax, table, cu_q, kv_lens, max_q, max_kv, causal, window, scale, rotate)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
        os_ = _strides2(q.shape[1] * q.shape[2], q.shape[2])
    else:
        os_ = _rows(out, "out", q.dtype, q.device)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    need = lib.nvfp4_kv_attention_workspace(q.shape[0], q.shape[1], ctypes.byref(c), ctypes.byref(b))
    if workspace is None:
        if need > 0 and stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        elif need > 0:
            with torch.cuda.stream(stream):  # the allocator ties the memory to the stream that uses it
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _buf(workspace, max(need, 0), torch.uint8, q.device, "workspace")
    fn = "nvfp4_kv_attention" if q.dtype == torch.bfloat16 else "nvfp4_kv_attention_f32"
    _check(fn, getattr(lib, fn)(_ptr(q), q.shape[0], q.shape[1], qs, ctypes.byref(c), ctypes.byref(b), _ptr(out),
                                os_, _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                _stream(q.device, stream)))
    return out
