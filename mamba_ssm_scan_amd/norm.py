"""The joint between two blocks of a hybrid stack: residual, gate, scale and the norms on either side, with gradients.

torch tensors in, the C entry points of include/m3_norm.h called, as in `binding`: argument marshalling only, outputs
and workspaces allocated with torch on the call's stream, no other implementation behind it.

    y = norm.residual_norm(x, weight=w)                          # the first block's input: the stream's norm
    o = block(y)
    x, y = norm.residual_norm(x, o, weight=w2)                   # x + o, and the next block's input
    x, y = norm.residual_norm(x, o, gate=g, scale=s, post_weight=w1, weight=w2)   # o normed, gated, scaled
    x = norm.residual_norm(x, o)                                 # after the last block
"""
from __future__ import annotations

import ctypes
import warnings
from typing import Optional

import torch

from . import binding
from .attention import _complain, _dense, _device_of, _handle, _no_tangents, _on_stream
from .binding import check

GATES = {"identity": 0, "silu": 1, "sigmoid": 2}

# every symbol include/m3_norm.h declares
EXPORTS = ["m3_residual_norm", "m3_residual_norm_backward", "m3_residual_norm_backward_workspace_size"]

_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class M3Lines(ctypes.Structure):
    _fields_ = [("p", _vp), ("stride", _i64)]


class M3Joint(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("width", _i32), ("stream_dtype", _i32), ("io_dtype", _i32),
                ("gate_fn", _i32), ("eps", _f32), ("factor", _f32), ("scale", _vp), ("post_weight", _vp), ("weight", _vp)]


_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = binding.load()
        joint, lines = ctypes.POINTER(M3Joint), ctypes.POINTER(M3Lines)
        lib.m3_residual_norm.argtypes = [joint] + [lines] * 5 + [_vp]
        lib.m3_residual_norm.restype = ctypes.c_int
        lib.m3_residual_norm_backward.argtypes = [joint] + [lines] * 8 + [_vp] * 4 + [_sz, _vp]
        lib.m3_residual_norm_backward.restype = ctypes.c_int
        lib.m3_residual_norm_backward_workspace_size.argtypes = [joint, _i32]
        lib.m3_residual_norm_backward_workspace_size.restype = _sz
        _ready = lib
    return _ready


def _lines(t, name: str, device, dtype, shape) -> Optional[M3Lines]:
    """Rows [..., width] where they lie: the entries of a row contiguous, the rows at one stride."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device or t.shape != shape:
        _complain(t, name, device, dtype, shape)
    if t.is_contiguous():
        return M3Lines(t.data_ptr(), shape[-1])
    if t.dim() == 2:
        st = t.stride()
        if st[1] != 1 and shape[1] > 1:
            raise ValueError(f"{name}: the entries of a row must be contiguous")
        return M3Lines(t.data_ptr(), st[0])
    try:
        rows = t.detach().view(-1, shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: its rows must lie at one stride") from None
    return _lines(rows, name, device, dtype, rows.shape)


def _empty(like: torch.Tensor, dtype) -> torch.Tensor:
    """A dense tensor of this shape (torch's quickest call for it)."""
    return torch.empty_like(like) if like.dtype is dtype and like.is_contiguous() else like.new_empty(like.shape, dtype=dtype)


def _joint(x_dtype, o_dtype, x, device, gate_fn, scale, post_weight, weight, eps) -> M3Joint:
    shape = x.shape
    if not shape:
        raise ValueError("rows must be [..., width]")
    W = shape[-1]
    fn = GATES.get(gate_fn)
    if fn is None:
        raise ValueError(f"unknown gate_fn {gate_fn!r}: {', '.join(GATES)}")
    factor, vec, each = 1.0, None, (W,)
    if isinstance(scale, torch.Tensor):
        vec = _dense(scale, "scale", device, torch.float32, each)
    elif scale is not None:
        factor = float(scale)
    pw = None if post_weight is None else _dense(post_weight, "post_weight", device, torch.float32, each)
    w = None if weight is None else _dense(weight, "weight", device, torch.float32, each)
    return M3Joint(x.numel() // W if W else 0, W, binding._io_code(x_dtype), binding._io_code(o_dtype), fn, eps, factor, vec,
                   pw, w)


class _ResidualNorm(torch.autograd.Function):
    """residual_norm as a step of autograd; the gradients are not differentiable again."""

    @staticmethod
    def forward(ctx, x, o, gate, scale, post_weight, weight, gate_fn, eps, dtype):
        ctx.set_materialize_grads(False)
        vec = scale if isinstance(scale, torch.Tensor) else None
        got = _forward(x, o, gate, gate_fn, scale, post_weight, weight, eps, None, dtype)
        h = x if o is None else got[0] if weight is not None else got
        ctx.save_for_backward(h if weight is not None else None, o, gate, vec, post_weight, weight)
        ctx.how = (gate_fn, eps, scale if vec is None else None)
        return got

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        h, o, gate, scale, post_weight, weight = ctx.saved_tensors
        gate_fn, eps, factor = ctx.how
        dh = grads[0] if o is not None else None
        dy = grads[-1] if weight is not None else None
        if dh is None and dy is None:
            return (None,) * 9
        # (a sum's gradient has no strides, a broadcast one's rows not one stride)
        rows = lambda t: t if t is None or (t.dim() == 2 and t.stride(1) == 1) else t.contiguous()  # noqa: E731
        need = ctx.needs_input_grad
        g = residual_norm_backward(rows(dh), rows(dy), h if dy is not None else None, o, gate=gate, gate_fn=gate_fn,
                                   scale=factor if scale is None else scale, post_weight=post_weight,
                                   weight=weight if dy is not None else None, eps=eps,
                                   want=[k for k, n in zip(_GRADS, need) if n and not (k == "weight" and dy is None)])
        return tuple(g[k] for k in _GRADS) + (None, None, None)


_GRADS = ("x", "o", "gate", "scale", "post_weight", "weight")


def _no_graph_through(out, x, asked: bool):
    """Refuses an `out` that autograd would go on taking for what it held before, or whose h would stand for an x that has
    no o in it; says so where a gradient that is asked for ends at an `out` of its own."""
    if not isinstance(out, torch.Tensor):
        return
    if out.requires_grad or (asked and (out is x or (out.numel() > 0 and out.data_ptr() == x.data_ptr()))):
        raise RuntimeError("out takes no part in autograd: it may neither require a gradient nor, where an input does, be "
                           "x itself (torch.no_grad() where none is wanted)")
    if asked:
        warnings.warn("residual_norm: the results take no part in autograd, as out is given (torch.no_grad() says that "
                      "none is wanted)", stacklevel=5)


@_on_stream
def _forward(x, o, gate, gate_fn, scale, post_weight, weight, eps, out, dtype):
    dev = _device_of(x, "x")
    if o is None and (gate is not None or out is not None):
        raise ValueError("gate or out without o")
    _no_tangents("residual_norm", x, o, gate, scale, post_weight, weight)
    if torch.is_grad_enabled():
        asked = False
        for t in (x, o, gate, scale, post_weight, weight):
            if isinstance(t, torch.Tensor) and t.requires_grad:
                asked = True
                break
        if out is not None:
            _no_graph_through(out, x, asked)
        elif asked:
            return _ResidualNorm.apply(x, o, gate, scale, post_weight, weight, gate_fn, eps, dtype)
    shape, xt = x.shape, x.dtype
    ot = getattr(o, "dtype", None) if o is not None else xt if dtype is None else dtype
    if dtype is not None and dtype is not ot:
        raise ValueError(f"dtype {dtype} beside an o of {ot}")
    j = _joint(xt, ot, x, dev, gate_fn, scale, post_weight, weight, eps)
    rx = _lines(x, "x", dev, xt, shape)
    ro = rg = rh = ry = h = y = None
    if o is not None:
        ro = _lines(o, "o", dev, ot, shape)
        rg = _lines(gate, "gate", dev, ot, shape)
        if out is None:
            h = _empty(x, xt)
            rh = M3Lines(h.data_ptr(), shape[-1])
        else:
            h, rh = out, _lines(out, "out", dev, xt, shape)
    if weight is not None:
        y = _empty(x, ot)
        ry = M3Lines(y.data_ptr(), shape[-1])
    check(_lib().m3_residual_norm(j, rx, ro, rg, rh, ry, _handle(dev)))
    if out is not None:  # what autograd kept of it before is no longer there
        torch.autograd.graph.increment_version(out)
    return y if o is None else h if weight is None else (h, y)


def residual_norm(x, o=None, *, gate=None, gate_fn: str = "silu", scale=None, post_weight=None, weight=None,
                  eps: float = 1e-6, out=None, dtype=None, stream=None):
    """m3_residual_norm: h = x + scale * a(gate) * N(o; post_weight) and y = N(h; weight); returns (h, y), h alone
    without weight, or y = N(x; weight) alone without o.

    x [..., width] the residual stream (fp32 or bf16), o and gate of its shape (bf16, or fp32 beside an fp32 stream);
    parts of a fused projection are used where they lie. gate_fn: "silu", "sigmoid" or "identity". scale: fp32
    [width] or a number. post_weight, weight: fp32 [width]; without post_weight o is not normed. Norms are of the
    root mean square, N(v; w) = v w / sqrt(mean v^2 + eps). width: up to 8192. out: where h goes, may be x itself.
    dtype: y's type without o (x's unless given; with o it is o's). stream: the current one unless given. The results
    take part in autograd where an input does (as in torch, a backward pass is captured into a graph only while no eager
    graph of the same leaves lives). With out they take no part, which is said by a warning where an input requires a
    gradient; an out that requires one, or that is then x itself, is refused (both hold while gradients are recorded). Inputs
    with tangents of forward-mode differentiation are refused.
    """
    return _forward(x, o, gate, gate_fn, scale, post_weight, weight, eps, out, dtype, stream=stream)


@_on_stream
def _backward(first, dh, dy, h, o, gate, gate_fn, scale, post_weight, weight, eps, want):
    dev, shape = first.device, first.shape
    xt = h.dtype if h is not None else dh.dtype
    ot = o.dtype if o is not None else dy.dtype
    j = _joint(xt, ot, first, dev, gate_fn, scale, post_weight, weight, eps)
    given = {"x": True, "o": o is not None, "gate": gate is not None, "scale": o is not None and j.scale,
             "post_weight": o is not None and j.post_weight, "weight": j.weight}
    ins = [_lines(t, n, dev, d, shape) for t, n, d in ((dh, "dh", xt), (dy, "dy", ot), (h, "h", xt), (o, "o", ot),
                                                       (gate, "gate", ot))]
    g = dict.fromkeys(_GRADS)
    for k in _GRADS if want is None else want:
        if k not in given:
            raise ValueError(f"no gradient {k!r}: {', '.join(_GRADS)}")
        if given[k]:
            g[k] = (_empty(first, xt if k == "x" else ot) if k in ("x", "o", "gate") else
                    first.new_empty(shape[-1], dtype=torch.float32))
    if all(t is None for t in g.values()):
        return g
    outs = [_lines(g[k], "d" + k, dev, xt if k == "x" else ot, shape) for k in ("x", "o", "gate")]
    sums = [None if g[k] is None else g[k].data_ptr() for k in ("weight", "post_weight", "scale")]
    lib = _lib()
    n = lib.m3_residual_norm_backward_workspace_size(j, any(p is not None for p in sums))
    ws = first.new_empty(n, dtype=torch.uint8) if n else None
    check(lib.m3_residual_norm_backward(j, *ins, *outs, *sums, ws.data_ptr() if n else None, n, _handle(dev)))
    return g


def residual_norm_backward(dh, dy, h, o=None, *, gate=None, gate_fn: str = "silu", scale=None, post_weight=None,
                           weight=None, eps: float = 1e-6, want=None, stream=None):
    """m3_residual_norm_backward: the gradients at stream h (the h that residual_norm returned; x without o), as a
    dict with the keys x, o, gate (rows), scale, post_weight, weight (fp32 [width]); None where there is no such input.

    dh, dy: the gradients of h and y, of their types; either may be None (dy without weight). Without dy, h is not
    needed. want: the keys to form, all unless given. stream: the current one unless given.
    """
    if (dy is None) != (weight is None):
        raise ValueError("dy and weight must be given together")
    if dh is None and dy is None:
        raise ValueError("neither dh nor dy is given")
    if dy is not None and h is None:
        raise ValueError("dy without h")
    _no_tangents("residual_norm_backward", dh, dy, h, o, gate, scale, post_weight, weight)
    first = dh if dh is not None else dy
    _device_of(first, "dh" if dh is not None else "dy")
    return _backward(first, dh, dy, h if dy is not None else None, o, gate, gate_fn, scale, post_weight, weight, eps, want,
                     stream=stream)
