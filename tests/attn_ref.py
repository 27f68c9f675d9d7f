"""The attention layer's definitions in 64 bits (CPU), for the tests: rotation, the block codes of the cache, attention."""
import math

import torch

BLOCK = 16
TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def turn(x, positions, inv_freq, interleaved=False, mscale=1.0, backward=False):
    """x [tokens][heads][dim] turned, as a complex product per pair."""
    half = inv_freq.numel()
    x = x.double()
    if not x.numel():
        return x
    head, tail = x[..., :2 * half], x[..., 2 * half:]
    z = head.unflatten(-1, (half, 2)) if interleaved else head.unflatten(-1, (2, half)).transpose(-1, -2)
    th = positions.double()[:, None, None] * inv_freq.double()
    w = torch.polar(torch.full_like(th, mscale), -th if backward else th)
    y = torch.view_as_real(torch.view_as_complex(z.contiguous()) * w)
    y = y.flatten(-2) if interleaved else y.transpose(-1, -2).flatten(-2)
    return torch.cat([y, tail], -1)


def nearest(x, dtype):
    """The nearest code's value, ties to even, held to the format's range."""
    if dtype == torch.int8:
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].double() - 4)
    return ((x / step).round() * step).clamp(-448, 448)


def step_of(x, dtype):
    """The distance between neighbouring codes at x (in units of the scale)."""
    if dtype == torch.int8:
        return torch.ones_like(x)
    return torch.exp2(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].double() - 4)


class Cache:
    """What a sequence of appends should hold: per sequence and head, values and scales by position, in 64 bits."""

    def __init__(self, batch, heads, dim, room, dtype):
        self.dtype, self.top = dtype, TOP[dtype]
        self.k, self.v = (torch.zeros(batch, room, heads, dim, dtype=torch.float64) for _ in range(2))
        self.ks, self.vs = (torch.zeros(batch, room // BLOCK, heads, dtype=torch.float64) for _ in range(2))

    def append(self, i, pos, k, v):
        """Rows k, v [n][heads][dim] (already turned) from position pos of sequence i."""
        for val, sc, new in ((self.k, self.ks, k.double()), (self.v, self.vs, v.double())):
            for blk in range(pos // BLOCK, (pos + new.shape[0] - 1) // BLOCK + 1 if new.shape[0] else 0):
                lo, hi = max(pos, blk * BLOCK), min(pos + new.shape[0], (blk + 1) * BLOCK)
                rows = new[lo - pos:hi - pos]
                old = val[i, blk * BLOCK:lo]
                s = rows.abs().amax((0, 2)) / self.top
                if lo > blk * BLOCK:
                    s = torch.maximum(s, sc[i, blk])
                s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)      # such a scale counts as 0
                u = torch.where(s > 0, s, torch.ones_like(s))[:, None]
                val[i, blk * BLOCK:lo] = nearest(old / u, self.dtype) * s[:, None]
                val[i, lo:hi] = nearest(rows / u, self.dtype) * s[:, None]
                sc[i, blk] = s


def attend(q, pos, k, v, scale, causal=True, window=0, seen=None):
    """One sequence: q [n][heads][dim] at positions pos [n] over k, v [len][kv heads][dim].

    Returns out, lse and, for error bounds, sum_j p_j |v_j| and the largest scale * sum |q| |k_j|."""
    n, H, D = q.shape
    L, G = k.shape[0], H // max(1, k.shape[1])
    there = torch.arange(L)
    ok = torch.ones(n, L, dtype=torch.bool) if seen is None else seen[None, :].expand(n, L).clone()
    if causal:
        ok &= there[None, :] <= pos[:, None]
    if window:
        ok &= there[None, :] > pos[:, None] - window
    qd, kd, vd = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    s = torch.matmul(qd.transpose(0, 1), kd.permute(1, 2, 0).contiguous()) * scale    # [H][n][L]
    big = torch.matmul(qd.abs().transpose(0, 1), kd.abs().permute(1, 2, 0).contiguous()) * abs(scale)
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(ok, (s - lse[..., None]).exp(), torch.zeros_like(s))
    p = torch.where(ok.any(-1)[None, :, None], p, torch.zeros_like(p))
    out, mag = torch.matmul(p, vd.transpose(0, 1)), torch.matmul(p, vd.abs().transpose(0, 1))
    top = big.masked_fill(~ok, 0.0).amax(-1) if L else torch.zeros(H, n, dtype=torch.float64)
    return out.transpose(0, 1), lse.transpose(0, 1), mag.transpose(0, 1), top.transpose(0, 1)


def attend_bound(out, mag, top, dim, length, io):
    """How far an output may be off, entry by entry.

    e: a score's fp32 error, (dim + 4) roundings of at most top, and the sums over `length` keys; a probability (and
    the sum it is divided by) then moves by at most 4 e relative. bf16 rows: each probability is rounded to 8 bits
    before the product with V (2^-8 of sum p |v|) and the output once (2^-8 of itself); fp32: 2^-23 instead."""
    e = 2.0 ** -24 * (length + (dim + 4) * top[..., None] + 8)
    r = 2.0 ** -8 if io == torch.bfloat16 else 2.0 ** -23
    return r * out.abs() + mag * (r * (1 + r) + 4 * e) + 1e-30
