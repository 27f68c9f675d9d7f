"""The attention layer of a hybrid stack: rotary positions, a paged 8-bit cache, attention over it.

torch tensors in, the C entry points of include/m3_attn.h called, as in `binding`: argument marshalling only,
outputs and workspaces allocated with torch on the call's stream, no other implementation behind it.
The cache's calls are for serving and take no part in autograd; `rope` does.

    cache = attention.KVCache.empty(num_pages, 64, kv_heads, head_dim)          # int8; or torch.float8_e4m3fn
    inv_freq, mscale = attention.rope_frequencies(head_dim)
    kv_len += 1                                                                  # int32 [batch], on the device
    q = cache.append(k, v, kv_len, pages, q=q, inv_freq=inv_freq)                # one new token a sequence
    o = cache.attend(q, kv_len, pages)

A prompt, or a ragged batch, gives its row offsets `cu_q` and, if it is known, the longest `max_q`.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch

from . import binding
from .binding import check

M3_KV_INT8, M3_KV_FP8 = 0, 1
BLOCK = 16  # tokens that share a scale, per head
FORMATS = {torch.int8: M3_KV_INT8, torch.float8_e4m3fn: M3_KV_FP8}

# every symbol include/m3_attn.h declares
EXPORTS = ["m3_rope", "m3_kv_append", "m3_kv_read", "m3_kv_attend", "m3_kv_attend_workspace_size"]

_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class M3KvCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("num_pages", _i64), ("page_size", _i32),
                ("heads", _i32), ("headdim", _i32), ("format", _i32)]


class M3KvBatch(ctypes.Structure):
    _fields_ = [("batch", _i64), ("tokens", _i64), ("max_pages", _i64), ("max_q", _i64), ("max_kv", _i64),
                ("cu_q", _vp), ("kv_len", _vp), ("pages", _vp)]


class M3Rows(ctypes.Structure):
    _fields_ = [("p", _vp), ("token_stride", _i64), ("head_stride", _i64)]


class M3Rotary(ctypes.Structure):
    _fields_ = [("inv_freq", _vp), ("rot", _i32), ("interleaved", _i32), ("mscale", _f32)]


_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = binding.load()
        cache, batch, rows, rot = (ctypes.POINTER(t) for t in (M3KvCache, M3KvBatch, M3Rows, M3Rotary))
        lib.m3_rope.argtypes = [rows, rows, _i64, _i32, _i32, ctypes.c_int, _vp, rot, _i32, _vp]
        lib.m3_kv_append.argtypes = [cache, batch, rows, rows, rows, rows, _i32, ctypes.c_int, rot, _vp]
        lib.m3_kv_read.argtypes = [cache, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp, ctypes.c_int, _vp]
        lib.m3_kv_attend.argtypes = [cache, batch, rows, _vp, _vp, _i32, ctypes.c_int, _f32, _i32, _i64, _vp, _sz, _vp]
        lib.m3_kv_attend_workspace_size.argtypes = [cache, batch, _i32, ctypes.c_int, _i32, _i64]
        lib.m3_kv_attend_workspace_size.restype = _sz
        for name in ("m3_rope", "m3_kv_append", "m3_kv_read", "m3_kv_attend"):
            getattr(lib, name).restype = ctypes.c_int
        _ready = lib
    return _ready


def _complain(t, name: str, device, dtype, shape):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dense(t: torch.Tensor, name: str, device, dtype, shape=None) -> int:
    """The address of a contiguous tensor of this device, type and shape."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device or (shape is not None
                                                                                         and t.shape != shape):
        _complain(t, name, device, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, device, dtype, shape=None) -> M3Rows:
    """[tokens][heads][dim] rows where they lie: the entries of a head contiguous, any other strides."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device or (shape is not None
                                                                                         and t.shape != shape):
        _complain(t, name, device, dtype, shape)
    st = t.stride()
    if len(st) != 3:
        raise ValueError(f"{name} must be [tokens][heads][dim]")
    if st[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the entries of a head must be contiguous")
    return M3Rows(t.data_ptr(), st[0], st[1])


def _device_of(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _on_stream(fn):
    """Runs a call on its device and stream: its allocations then belong to that stream, so that their memory is not
    handed on early. fn(..., stream=the raw handle)."""
    @functools.wraps(fn)
    def call(first, *args, stream=None, **kw):
        dev = getattr(first, "device", None)
        if stream is None:
            if dev is None or dev.type != "cuda" or dev.index == torch.cuda.current_device():
                return fn(first, *args, **kw)
            with torch.cuda.device(dev):
                return fn(first, *args, **kw)
        with torch.cuda.stream(stream):
            return fn(first, *args, **kw)
    return call


# the current stream's raw handle, without the Stream object around it where torch has that call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _rotary(inv_freq, device, interleaved, mscale) -> M3Rotary:
    p = _dense(inv_freq, "inv_freq", device, torch.float32)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rot / 2]")
    return M3Rotary(p, 2 * inv_freq.numel(), int(bool(interleaved)), float(mscale))


def rope_frequencies(rot: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                     trained_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(inv_freq [rot / 2] fp32, mscale): f_i = base^(-2i / rot), for contexts `factor` times the trained length.

    scaling None: as they are. "linear": f_i / factor (positions squeezed into the trained range). "base": the base
    grown by factor^(rot / (rot - 2)), so the slowest pair is squeezed by the factor and the fastest hardly. "bands":
    pairs that turn more than beta_fast times within trained_len keep f_i, those below beta_slow turns take
    f_i / factor, a linear blend between, and mscale = 0.1 ln(factor) + 1.
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and >= 2, got {rot}")
    if scaling not in (None, "linear", "base", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling is not None and not factor >= 1.0:
        raise ValueError(f"factor must be >= 1, got {factor}")
    if scaling == "base" and rot == 2:
        raise ValueError("scaling 'base' needs rot > 2")
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        if trained_len < 1 or not beta_fast > beta_slow:
            raise ValueError("scaling 'bands' needs trained_len >= 1 and beta_fast > beta_slow")
        turns = trained_len * f / (2.0 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    return f.to(torch.float32).to(device), mscale


class _Rope(torch.autograd.Function):
    """rope as a step of autograd: linear, with the transposed map as its gradient."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, interleaved, mscale, backward):
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = dict(interleaved=interleaved, mscale=mscale, backward=not backward)
        return rope(x.detach(), positions, inv_freq, interleaved=interleaved, mscale=mscale, backward=backward)

    @staticmethod
    def backward(ctx, dy):
        dy = dy if dy.stride(-1) == 1 or dy.shape[-1] == 1 else dy.contiguous()
        return rope(dy, *ctx.saved_tensors, **ctx.how), None, None, None, None, None


@_on_stream
def rope(x, positions, inv_freq, *, interleaved: bool = False, mscale: float = 1.0, backward: bool = False, out=None):
    """m3_rope: x [tokens][heads][dim] (bf16 or fp32) turned by positions [tokens] int32; returns out.

    backward: the transposed map (dL/dx from x = dL/dy). out may be x itself. stream: the current one unless given.
    The result takes part in autograd where x does, unless out is given.
    """
    dev, dt = _device_of(x, "x"), x.dtype
    if out is None and x.requires_grad and torch.is_grad_enabled():
        return _Rope.apply(x, positions, inv_freq, interleaved, mscale, backward)
    code = binding._io_code(dt)
    rx = _rows(x, "x", dev, dt)
    shape = x.shape
    T, H, D = shape
    pos = _dense(positions, "positions", dev, torch.int32, (T,))
    rot = _rotary(inv_freq, dev, interleaved, mscale)
    if out is None:
        out = x.new_empty(shape)
    ry = _rows(out, "out", dev, dt, shape)
    check(_lib().m3_rope(rx, ry, T, H, D, code, pos, rot, 1 if backward else 0, _handle(dev)))
    return out


class KVCache:
    """A paged cache of keys and values in 8 bits, one scale per 16 tokens and head (the layout of m3_kv_cache).

    k [pages][heads][page_size / 16][16][dim] and v [pages][heads][page_size / 16][dim][16], int8 or float8_e4m3fn;
    k_scale, v_scale [pages][heads][page_size / 16] fp32; all kept for good (other tensors are another KVCache).
    Sequences, page tables and lengths are the caller's: `pages` [batch][max_pages] int32 names each sequence's pages in
    order, `kv_len` [batch] int32 its tokens with the call's new ones in (0: an idle slot). Rows of the call's tokens
    follow one another, `cu_q` [batch + 1] int32 where a sequence may have other than one, `max_q` at least the longest
    (all rows unless given; the longest itself may be a fifth faster). Rows past `max_q` are left out, and what their
    outputs held stays.
    """

    def __init__(self, k, v, k_scale, v_scale):
        dev = _device_of(k, "k")
        if k.dtype not in FORMATS:
            raise TypeError(f"k must be int8 or float8_e4m3fn, got {k.dtype}")
        if k.dim() != 5 or k.shape[3] != BLOCK:
            raise ValueError("k must be [pages][heads][page_size / 16][16][dim]")
        P, H, S, _, D = k.shape
        _dense(k, "k", dev, k.dtype)
        _dense(v, "v", dev, k.dtype, (P, H, S, D, BLOCK))
        _dense(k_scale, "k_scale", dev, torch.float32, (P, H, S))
        _dense(v_scale, "v_scale", dev, torch.float32, (P, H, S))
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale
        self.device, self.heads, self.head_dim, self.page_size = dev, H, D, S * BLOCK
        self._c = M3KvCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), P, S * BLOCK, H, D,
                            FORMATS[k.dtype])
        self._sizes = {}  # workspace bytes by a call's sizes

    @classmethod
    def empty(cls, num_pages: int, page_size: int, heads: int, head_dim: int, dtype=torch.int8, device="cuda"):
        """A cache that holds nothing yet (its memory is not cleared: a block is written whole when it begins)."""
        if page_size < BLOCK or page_size % BLOCK:
            raise ValueError(f"page_size must be a power of two >= {BLOCK}, got {page_size}")
        sub = page_size // BLOCK
        new = lambda *shape: torch.empty(shape, dtype=torch.int8, device=device).view(dtype)  # noqa: E731
        scale = lambda: torch.empty((num_pages, heads, sub), dtype=torch.float32, device=device)  # noqa: E731
        return cls(new(num_pages, heads, sub, BLOCK, head_dim), new(num_pages, heads, sub, head_dim, BLOCK), scale(),
                   scale())

    # calls go to the tensors that the cache was made of: their contents may change, the tensors not
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)

    def _batch(self, tokens, kv_len, pages, cu_q, max_q, max_kv) -> M3KvBatch:
        dev = self.device
        lens, table = _dense(kv_len, "kv_len", dev, torch.int32), _dense(pages, "pages", dev, torch.int32)
        if kv_len.dim() != 1 or pages.dim() != 2 or pages.shape[0] != kv_len.shape[0]:
            raise ValueError("kv_len must be [batch] and pages [batch][max_pages]")
        b, room = pages.shape
        cu = None
        if cu_q is not None:
            cu = _dense(cu_q, "cu_q", dev, torch.int32, (b + 1,))
        elif tokens != b:
            raise ValueError(f"{tokens} rows for {b} sequences need cu_q")
        if max_q is None:
            max_q = 1 if cu is None else tokens
        return M3KvBatch(b, tokens, room, max_q, room * self.page_size if max_kv is None else max_kv, cu, lens, table)

    @_on_stream
    def append(self, k, v, kv_len, pages, *, cu_q=None, max_q: Optional[int] = None, q=None, q_out=None, inv_freq=None,
               interleaved: bool = False, mscale: float = 1.0):
        """m3_kv_append: k, v [tokens][heads][dim] (bf16 or fp32) into the cache, the keys turned by inv_freq (None:
        as they are). With q [tokens][q_heads][dim], returns it turned by the same positions. stream: the current one
        unless given."""
        dev, dt, T = self.device, k.dtype, k.shape[0]
        code = binding._io_code(dt)
        shape = (T, self.heads, self.head_dim)
        rk, rv = _rows(k, "k", dev, dt, shape), _rows(v, "v", dev, dt, shape)
        b = self._batch(T, kv_len, pages, cu_q, max_q, None)
        rot = None if inv_freq is None else _rotary(inv_freq, dev, interleaved, mscale)
        rq = ro = None
        qh = 0
        if q is not None:
            rq = _rows(q, "q", dev, dt)
            shape = q.shape
            qh = shape[1]
            if shape[0] != T or shape[2] != self.head_dim:
                raise ValueError(f"q has shape {tuple(shape)}, expected ({T}, q_heads, {self.head_dim})")
            if q_out is None:
                q_out = q.new_empty(shape)
            ro = _rows(q_out, "q_out", dev, dt, shape)
        elif q_out is not None:
            raise ValueError("q_out without q")
        check(_lib().m3_kv_append(self._c, b, rk, rv, rq, ro, qh, code, rot, _handle(dev)))
        return q_out

    @_on_stream
    def read(self, first, count, pages, max_count: int, dtype=torch.bfloat16):
        """m3_kv_read: the values held at positions first[i] .. first[i] + count[i] - 1 of each sequence, as k, v
        [batch][max_count][heads][dim]; rows past count are zero. stream: the current one unless given."""
        dev = self.device
        code = binding._io_code(dtype)
        at = _dense(first, "first", dev, torch.int32)
        b = first.numel()
        n, table = _dense(count, "count", dev, torch.int32, (b,)), _dense(pages, "pages", dev, torch.int32)
        if first.dim() != 1 or pages.dim() != 2 or pages.shape[0] != b:
            raise ValueError("first and count must be [batch] and pages [batch][max_pages]")
        if max_count < 0:
            raise ValueError(f"max_count {max_count} < 0")
        shape = (b, max_count, self.heads, self.head_dim)
        k, v = first.new_empty(shape, dtype=dtype), first.new_empty(shape, dtype=dtype)
        check(_lib().m3_kv_read(self._c, b, at, n, table, pages.shape[1], max_count, k.data_ptr(), v.data_ptr(), code,
                                _handle(dev)))
        return k, v

    @_on_stream
    def attend(self, q, kv_len, pages, *, cu_q=None, max_q: Optional[int] = None, max_kv: Optional[int] = None,
               scale: Optional[float] = None, causal: bool = True, window: int = 0, out=None, lse=False):
        """m3_kv_attend: q [tokens][q_heads][dim] over the cache; returns out, or (out, lse) with lse=True.

        scale: 1 / sqrt(dim) unless given. causal: a row sees the keys up to its own position; window > 0: only the
        last `window` of them. A row that sees nothing gives 0 (and lse -inf). max_kv: at least the largest kv_len,
        the page table's room unless given. stream: the current one unless given.
        """
        dev, dt = self.device, q.dtype
        code = binding._io_code(dt)
        rq = _rows(q, "q", dev, dt)
        shape = q.shape
        T, H, D = shape
        if D != self.head_dim:
            raise ValueError(f"q has heads of {D} entries, the cache of {self.head_dim}")
        b = self._batch(T, kv_len, pages, cu_q, max_q, max_kv)
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        lib = _lib()
        if out is None:
            out = q.new_empty(shape)
        o = _dense(out, "out", dev, dt, shape)
        z = q.new_empty((T, H), dtype=torch.float32) if lse else None
        causal = 1 if causal else 0
        key = (b.batch, T, b.max_pages, b.max_q, b.max_kv, cu_q is None, H, code, causal, window)
        n = self._sizes.get(key)
        if n is None:
            if len(self._sizes) > 4096:
                self._sizes.clear()
            n = self._sizes[key] = lib.m3_kv_attend_workspace_size(self._c, b, H, code, causal, window)
        ws = q.new_empty(n, dtype=torch.uint8) if n else None
        check(lib.m3_kv_attend(self._c, b, rq, o, z.data_ptr() if lse else None, H, code, scale, causal, window,
                               ws.data_ptr() if n else None, n, _handle(dev)))
        return (out, z) if lse else out
