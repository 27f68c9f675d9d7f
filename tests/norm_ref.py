"""The joint between two blocks in 64 bits (CPU), for the tests, with bounds on what fp32 arithmetic may be off by.

u = 2^-24 is a rounding's half step. A sum over a row or over the rows is formed as a tree of short chains, so that a term
passes a bounded number of additions (SUM, for a row of 8192 and the rows of these tests); a mean's, a root's and a
product's few roundings are in it too. sigmoid is e^-|g| through a power of two (the argument's rounding: |g| u relative)
and a reciprocal of a few ulp; a power below 2^-126, the least normal number, is 0, so a sigmoid may be off by that much
whatever its size (LEAST), g sigmoid(g) and the slopes by (1 + |g|) times as much."""
import torch

U = 2.0 ** -24
LEAST = 2.0 ** -126
SUM = 80
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gate_parts(fn, g):
    """a(g), a'(g), and the size of what a' is added from."""
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)
    if fn == "identity":
        return g, torch.ones_like(g), torch.ones_like(g)
    if fn == "sigmoid":
        return s, s * rest, s * rest
    return g * s, s + g * s * rest, s + (g * s * rest).abs()


def norm(v, w, eps):
    r = (v.square().mean(-1, keepdim=True) + eps).rsqrt()
    return v * r * w, r


def forward(x, o, gate, fn, scale, pw, w, eps):
    """h, y and the bounds of their errors before the output's rounding (dicts by name)."""
    d = lambda t: t if t is None or isinstance(t, float) else t.double()  # noqa: E731
    x, o, gate, scale, pw, w = (d(t) for t in (x, o, gate, scale, pw, w))
    got, bound = {}, {}
    h, dh = x, torch.zeros_like(x)
    if o is not None:
        b = o if pw is None else norm(o, pw, eps)[0]
        few = torch.full_like(b, 2.0 * SUM if pw is not None else 8.0)
        lost = 0.0
        s = 1.0 if scale is None else scale
        if gate is not None:
            lost = (b * s * (1 + gate.abs())).abs() * LEAST
            b = b * gate_parts(fn, gate)[0]
            few = few + 8 + 2 * gate.abs()
        b = b * s
        h = x + b
        dh = (b.abs() * few + h.abs()) * U + lost
        got["h"], bound["h"] = h, dh
    if w is not None:
        y, r = norm(h, w, eps)
        rel = dh.square().sum(-1, keepdim=True).sqrt() / h.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-300)
        got["y"], bound["y"] = y, (w * r).abs() * dh + y.abs() * (2 * SUM * U + rel)
    return got, bound


def backward(dh, dy, h, o, gate, fn, scale, pw, w, eps):
    """The gradients by their formulas, and bounds as above."""
    d = lambda t: t if t is None or isinstance(t, float) else t.double()  # noqa: E731
    dh, dy, h, o, gate, scale, pw, w = (d(t) for t in (dh, dy, h, o, gate, scale, pw, w))
    got, bound = {}, {}
    like = dh if dh is not None else dy
    t = torch.zeros_like(like) if dh is None else dh
    err = torch.zeros_like(t)
    rows = like.shape[0]
    few = SUM + rows / 256
    if w is not None:
        r = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
        n, u = h * r, dy * w
        t = t + r * (u - n * (u * n).mean(-1, keepdim=True))
        size = (0.0 if dh is None else dh.abs()) + r * (u.abs() + n.abs() * (u * n).abs().mean(-1, keepdim=True))
        err = size * 4 * SUM * U
        got["weight"] = (dy * n).sum(0)
        bound["weight"] = (dy * n).abs().sum(0) * (2 * SUM + few) * U
    got["x"], bound["x"] = t, err
    if o is None:
        return got, bound
    one = torch.ones_like(o)
    act, slope, slope_size = (one, one, one) if gate is None else gate_parts(fn, gate)
    s = one if scale is None else scale
    soft = 16 + (0 if gate is None else 4 * gate.abs())
    lost = torch.zeros_like(o) if gate is None else (1 + gate.abs()) * LEAST
    r1 = torch.ones_like(o[..., :1]) if pw is None else (o.square().mean(-1, keepdim=True) + eps).rsqrt()
    n1, p = o * r1, one if pw is None else pw
    v = t * act * s
    dv = (act * s).abs() * err + v.abs() * soft * U + (t * s).abs() * lost
    if gate is not None:
        got["gate"] = t * s * slope * n1 * p
        bound["gate"] = (s * n1 * p).abs() * (slope_size.abs() * (err + t.abs() * (2 * SUM + soft) * U) + t.abs() * lost)
    if isinstance(scale, torch.Tensor):
        got["scale"] = (t * act * n1 * p).sum(0)
        bound["scale"] = ((n1 * p).abs() * (act.abs() * (err + t.abs() * (2 * SUM + soft + few) * U) + t.abs() * lost)).sum(0)
    if pw is None:
        got["o"], bound["o"] = v, dv
    else:
        got["post_weight"] = (v * n1).sum(0)
        bound["post_weight"] = (n1.abs() * (dv + v.abs() * (2 * SUM + few) * U)).sum(0)
        got["o"] = r1 * (v * p - n1 * (v * p * n1).mean(-1, keepdim=True))
        mean = (p * n1).abs() * (dv + v.abs() * 4 * SUM * U)
        bound["o"] = r1 * (p.abs() * (dv + v.abs() * 4 * SUM * U) + n1.abs() * mean.mean(-1, keepdim=True)
                           + n1.abs() * (v * p * n1).abs().mean(-1, keepdim=True) * 4 * SUM * U)
    return got, bound
