"""Timed cases of what joins a hybrid stack's layers, and of its attention layer under a window with sinks or a shared prefix.

The joint between two blocks: a block's output is normed, gated, scaled and added to the residual stream, whose norm is
the next block's input (and the gradients of that). Attention over the paged 8-bit cache: a sliding window beside first
tokens that stay visible, and sequences that hold the same first pages. Each case names its sizes; `prepare` draws its
inputs, `run` makes one pass, in plain torch operations in 32 bits or through the package's kernels (`own`), and `exact`
evaluates the definitions in 64 bits.

The cache holds tokens in pages of `page` tokens, each (page, head) as blocks of 16 tokens with one scale a block:
K codes [pages][heads][page / 16][16][dim], V codes [pages][heads][page / 16][dim][16], scales [pages][heads][page / 16];
a value is its code times its block's scale. Sequence i holds its tokens in the pages `pages[i]` names, in order; the
sequences of a group hold their first `count` pages together, named by the group's own table.
"""
import math
import random

import torch

own = False

BLOCK = 16                                   # tokens that share a scale
CODE = {"int8": (torch.int8, 127.0), "fp8": (torch.float8_e4m3fn, 448.0)}
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one step of a batch of 128 between two blocks: a plain residual, the next block's norm; only the launch counts
        dict(name="joint_step_b128", op="joint", pass_="forward", io="bf16", res="bf16", tokens=128, width=2048,
             post=False, gate="", scale=False, pre=True),
        # a training batch of 4 sequences of 2048 tokens, the stream in 32 bits, norms on both sides, gate and scale
        dict(name="joint_forward_4x2048", op="joint", pass_="forward", io="bf16", res="f32", tokens=8192, width=2048,
             post=True, gate="silu", scale=True, pre=True),
        # the gradients of that batch, the stream in 16 bits
        dict(name="joint_backward_4x2048", op="joint", pass_="backward", io="bf16", res="bf16", tokens=8192, width=2048,
             post=True, gate="silu", scale=True, pre=True),
        # a 32-bit check of a ragged batch at an odd width, no scale
        dict(name="joint_backward_f32_odd", op="joint", pass_="backward", io="f32", res="f32", tokens=1999, width=1283,
             post=True, gate="sigmoid", scale=False, pre=True),
        # a larger step of training as autograd runs it: forward and backward
        dict(name="joint_train_16384x4096", op="joint", pass_="train", io="bf16", res="f32", tokens=16384, width=4096,
             post=True, gate="silu", scale=True, pre=True),
        # one long conversation whose old pages are given back, one token
        dict(name="sinks_one_ctx30000", op="attend", fmt="int8", io="bf16", batch=1, q_lo=1, q_hi=1, ctx_lo=30000,
             ctx_hi=30000, idle=0, heads=16, kv=4, dim=128, page=64, window=1024, sinks=4, lse=False),
        # a serving batch of 128 at many lengths, within and beyond the window
        dict(name="sinks_step_b128", op="attend", fmt="int8", io="bf16", batch=128, q_lo=1, q_hi=1, ctx_lo=127,
             ctx_hi=16383, idle=3, heads=16, kv=4, dim=128, page=64, window=2048, sinks=64, lse=True),
        # two prompts of 8192 tokens, each row under its window
        dict(name="sinks_prompt_2x8192", op="attend", fmt="fp8", io="bf16", batch=2, q_lo=8192, q_hi=8192, ctx_lo=0,
             ctx_hi=0, idle=0, heads=16, kv=4, dim=128, page=64, window=1024, sinks=16, lse=False),
        # 16 answers to one prompt of 8192 tokens, a step each
        dict(name="prefix_step_b16", op="attend", fmt="int8", io="bf16", batch=16, q_lo=1, q_hi=1, ctx_lo=1,
             ctx_hi=511, idle=0, heads=16, kv=4, dim=128, page=64, window=0, sinks=0, groups=1, pre_lo=128, pre_hi=128,
             lse=False),
        # a serving batch of 128 behind one long system prompt
        dict(name="prefix_step_b128", op="attend", fmt="fp8", io="bf16", batch=128, q_lo=1, q_hi=1, ctx_lo=63,
             ctx_hi=1023, idle=2, heads=16, kv=4, dim=128, page=64, window=0, sinks=0, groups=1, pre_lo=128,
             pre_hi=128, lse=False),
        # 32-bit drafts of a few tokens in groups with prefixes of their own, small pages, odd lengths, idle slots
        dict(name="prefix_draft_f32_groups", op="attend", fmt="int8", io="f32", batch=23, q_lo=0, q_hi=5, ctx_lo=0,
             ctx_hi=301, idle=2, heads=6, kv=3, dim=80, page=16, window=0, sinks=0, groups=5, pre_lo=3, pre_hi=61,
             lse=True),
        # 8 questions of 256 tokens on one document of 16384
        dict(name="prefix_questions_8x256", op="attend", fmt="fp8", io="bf16", batch=8, q_lo=256, q_hi=256, ctx_lo=0,
             ctx_hi=0, idle=0, heads=16, kv=4, dim=128, page=64, window=0, sinks=0, groups=1, pre_lo=256, pre_hi=256,
             lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["joint", "attend", "attend"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "joint":
        pass_ = rng.choice(["forward", "forward", "backward", "backward", "train"])
        width = _log(rng, 64, 8192)
        width = width if rng.random() < 0.3 else max(64, width // 64 * 64)
        tokens = min(_log(rng, 1, 16384), ((1 << 26) if io == "bf16" else (1 << 25)) // width)
        return dict(op=op, pass_=pass_, io=io, res="f32" if io == "f32" else rng.choice(["bf16", "f32"]), tokens=tokens,
                    width=width, post=rng.random() < 0.6, gate=rng.choice(["", "silu", "sigmoid", "identity"]),
                    scale=rng.random() < 0.5, pre=pass_ != "forward" or rng.random() < 0.85)
    dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 6, 8])
    fmt = rng.choice(["int8", "fp8"])
    page = rng.choice([16, 32, 64, 128])
    c = dict(op=op, fmt=fmt, io=io, heads=heads, kv=kv, dim=dim, page=page, window=0, sinks=0, lse=rng.random() < 0.3)
    kind = rng.choice(["step", "step", "draft", "rows"])
    q_hi = {"step": 1, "draft": rng.randint(2, 9), "rows": _log(rng, 10, 2048)}[kind]
    if rng.random() < 0.45:     # a window beside first tokens
        c.update(window=_log(rng, 1, 4096), sinks=_log(rng, 1, 300))
        ctx_hi = _log(rng, 1, 30000) if kind != "rows" or rng.random() < 0.5 else 0
        room = ctx_hi + q_hi
        most = 130
    else:
        pre_hi = _log(rng, 1, 16384 // page)
        ctx_hi = _log(rng, 1, 1500) - 1
        q_hi = min(q_hi, 512)
        room = ctx_hi + q_hi + pre_hi * page
        most = 130 if kind in ("step", "draft") else 8
    batch = max(1, min(_log(rng, 1, most), (1 << 29) // ((room + page) * kv * dim), (1 << 28) // (room * heads * q_hi)))
    q_hi = max(1, min(q_hi, (1 << 28) // (room * heads)))
    if not c["window"]:
        groups = min(batch, _log(rng, 1, 8))
        c.update(groups=groups, pre_lo=rng.choice([pre_hi, max(0, pre_hi // 3)]), pre_hi=pre_hi)
    c.update(batch=batch, q_lo=rng.choice([q_hi, q_hi, max(0, q_hi // 2)]) if q_hi > 1 else 1, q_hi=q_hi,
             ctx_lo=rng.choice([ctx_hi, ctx_hi // 3]), ctx_hi=ctx_hi, idle=min(rng.choice([0, 0, 1]), batch - 1))
    return c


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi (the first is hi), spread by the multiples of an irrational number."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * (((i + 1) * step) % 1.0)) for i in range(n)]


def _lengths(c):
    """(new tokens, tokens held after the call) of each sequence, (first sequence of each group and the end), (pages of
    each group's prefix); idle slots hold none and still bring a query row."""
    n = _spread(c["q_lo"], c["q_hi"], c["batch"], 0.7548776662466927)
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["batch"], 0.6180339887498949)
    cu, count = [0, c["batch"]], [0]
    if c.get("groups"):
        cu = [i * c["batch"] // c["groups"] for i in range(c["groups"] + 1)]
        count = _spread(c["pre_lo"], c["pre_hi"], c["groups"], 0.5698402909980532)
    held = [0] * c["batch"]
    for a, b, k in zip(cu, cu[1:], count):
        for i in range(a, b):
            held[i] = n[i] + ctx[i] + k * c["page"]
    for i in range(c["idle"]):
        held[c["batch"] - 1 - i] = 0
    return n, held, cu, count


# ---------------------------------------------------------------------------------------------------------- inputs

def _fill_pool(c, num_pages, gen, dev):
    """A cache in use: values with a spread of magnitudes by channel, as codes and scales."""
    dt, top = CODE[c["fmt"]]
    shape = (num_pages, c["kv"], c["page"] // BLOCK, BLOCK, c["dim"])
    pool = {}
    for name in ("k", "v"):
        channel = torch.exp(0.5 * torch.randn(c["dim"], generator=gen, device=dev)) if name == "k" else 1.0
        codes, scales = [], []
        for at in range(0, num_pages, 1024):
            x = torch.randn((min(1024, num_pages - at),) + shape[1:], generator=gen, device=dev) * channel
            s = x.abs().amax((-1, -2)) / top
            x = x / s[..., None, None]
            x = x.round() if c["fmt"] == "int8" else x
            x = x if name == "k" else x.transpose(-1, -2).contiguous()
            codes.append(x.clamp(-top, top).to(dt))
            scales.append(s)
        pool[name], pool[name + "_scale"] = torch.cat(codes), torch.cat(scales)
    return pool


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(dtype, *shape, size=1.0):
        return (size * torch.randn(shape, generator=gen, device=dev)).to(dtype)

    io = IO[c["io"]]
    if c["op"] == "joint":
        T, W, f32 = c["tokens"], c["width"], torch.float32
        s = dict(c=c, o=normal(io, T, W), gate=normal(io, T, W) if c["gate"] else None,
                 scale=0.5 + 0.1 * normal(f32, W) if c["scale"] else None,
                 post_weight=1.0 + 0.2 * normal(f32, W) if c["post"] else None,
                 weight=1.0 + 0.2 * normal(f32, W) if c["pre"] else None)
        s["h" if c["pass_"] == "backward" else "x"] = normal(IO[c["res"]], T, W, size=3.0)
        if c["pass_"] != "forward":
            s["dh"], s["dy"] = normal(IO[c["res"]], T, W), normal(io, T, W)
        return s
    n, held, cu_seqs, count = _lengths(c)
    page, batch = c["page"], c["batch"]
    max_pages = max(1, max(-(-h // page) for h in held))
    group = [g for g in range(len(count)) for _ in range(cu_seqs[g], cu_seqs[g + 1])]
    need = [range(count[group[i]], -(-h // page)) for i, h in enumerate(held)]          # pages of the sequence's own
    if c["window"]:             # of those, the pages that hold first tokens or some row's window
        need = [[j for j in r if j * page < c["sinks"] or (j + 1) * page > h - k - c["window"] + 1]
                for r, k, h in zip(need, n, held)]
    order = torch.randperm(sum(count) + sum(len(r) for r in need) + 3, generator=gen, device=dev).to(torch.int32).tolist()
    shared = [[order.pop() for _ in range(k)] for k in count]
    table = []
    for i, r in enumerate(need):
        row = (shared[group[i]] + [-1] * max_pages)[:max_pages]
        for j in r:
            row[j] = order.pop()
        table.append(row)
    wide = max(1, max(count))
    cu = [0]
    for k in n:
        cu.append(cu[-1] + k)
    num_pages = sum(count) + sum(len(r) for r in need) + 3
    ints = dict(dtype=torch.int32, device=dev)
    s = dict(c=c, pages=torch.tensor(table, **ints), kv_len=torch.tensor(held, **ints), cu_q=torch.tensor(cu, **ints),
             max_q=max(1, max(n)), max_kv=max(1, max(held)), q=normal(io, cu[-1], c["heads"], c["dim"]),
             shared=torch.tensor([(r + [0] * wide)[:wide] for r in shared], **ints),
             count=torch.tensor(count, **ints), cu_seqs=torch.tensor(cu_seqs, **ints),
             each_one=n == [1] * batch, **_fill_pool(c, num_pages, gen, dev))
    return s


# ---------------------------------------------------------------------------------------------------------- plain forms

def _gate(kind, g):
    """a(g) and its derivative."""
    if not kind:
        return None, None
    if kind == "identity":
        return g, torch.ones_like(g)
    sig = 1.0 / (1.0 + (-g).exp())
    if kind == "sigmoid":
        return sig, sig * (1.0 - sig)
    return g * sig, sig * (1.0 + g * (1.0 - sig))


def _times(x, *factors):
    for f in factors:
        x = x if f is None else x * f
    return x


def _plain_forward(s):
    c = s["c"]
    x, o = s["x"].float(), s["o"].float()
    if s["post_weight"] is not None:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["post_weight"]
    act = None if s["gate"] is None else _gate(c["gate"], s["gate"].float())[0]
    h = x + _times(o, act, s["scale"])
    out = {"h": h.to(s["x"].dtype)}
    if s["weight"] is not None:
        out["y"] = (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]).to(s["o"].dtype)
    return out


def _plain_backward(s, h):
    c = s["c"]
    io, res = s["o"].dtype, s["dh"].dtype
    h, o, t, dy = h.float(), s["o"].float(), s["dh"].float(), s["dy"].float()
    out = {}
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n, u = h * r, dy * s["weight"]
    t = t + r * (u - n * (u * n).mean(-1, keepdim=True))
    out["dweight"] = (dy * n).sum(0)
    out["dx"] = t.to(res)
    act, slope = _gate(c["gate"], None if s["gate"] is None else s["gate"].float())
    r1 = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) if s["post_weight"] is not None else None
    normed = _times(o, r1, s["post_weight"])
    v = _times(t, act, s["scale"])
    if act is not None:
        out["dgate"] = _times(t * normed * slope, s["scale"]).to(io)
    if s["scale"] is not None:
        out["dscale"] = _times(t * normed, act).sum(0)
    if r1 is not None:
        n1, vw = o * r1, v * s["post_weight"]
        out["dpost_weight"] = (v * n1).sum(0)
        v = r1 * (vw - n1 * (vw * n1).mean(-1, keepdim=True))
    out["do"] = v.to(io)
    return out


def _dense(s, pos, seq):
    """The values the cache holds at positions pos of sequences seq (both of one shape), [...][heads][dim] in 32 bits."""
    page = s["c"]["page"]
    group = torch.searchsorted(s["cu_seqs"][1:].long(), seq, right=True)
    at = pos // page
    pg = s["pages"].long()[seq, at.clamp(max=s["pages"].shape[1] - 1)]
    first = s["shared"].long()[group, at.clamp(max=s["shared"].shape[1] - 1)]
    pg = torch.where(at < s["count"][group], first, pg).clamp(min=0)
    sub, slot = pos % page // BLOCK, pos % BLOCK
    k = s["k"].view(torch.int8)[pg, :, sub, slot].view(s["k"].dtype).float() * s["k_scale"][pg, :, sub][..., None]
    v = s["v"].view(torch.int8)[pg, :, sub, :, slot].view(s["v"].dtype).float() * s["v_scale"][pg, :, sub][..., None]
    return k, v


def _plain_attend(s):
    c = s["c"]
    dev, group = s["q"].device, c["heads"] // c["kv"]
    t = torch.arange(s["q"].shape[0], device=dev)
    cu = s["cu_q"].long()
    seq = torch.searchsorted(cu[1:], t, right=True)
    row = t - cu[seq]
    pos = s["kv_len"].long()[seq] - (cu[1:] - cu[:-1])[seq] + row
    q = torch.zeros((c["batch"], s["max_q"], c["kv"], group, c["dim"]), device=dev)
    q[seq, row] = s["q"].float().view(-1, c["kv"], group, c["dim"]) / math.sqrt(c["dim"])
    at = torch.arange(s["max_kv"], device=dev).expand(c["batch"], -1)
    k, v = _dense(s, at, torch.arange(c["batch"], device=dev)[:, None].expand_as(at))
    place = torch.full((c["batch"], s["max_q"]), -1, device=dev)
    place[seq, row] = pos
    seen = (at[:, None, :] < s["kv_len"].long()[:, None, None]) & (at[:, None, :] <= place[..., None])
    if c["window"]:
        seen = seen & ((at[:, None, :] > place[..., None] - c["window"]) | (at[:, None, :] < c["sinks"]))
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, group, -1).reshape(c["batch"], 1, -1, s["max_kv"])
    w = q.permute(0, 2, 1, 3, 4).reshape(c["batch"], c["kv"], -1, c["dim"]) @ k.permute(0, 2, 3, 1).contiguous()
    w = w.masked_fill(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = (w - top.clamp(min=-3.0e38)).exp()
    total = w.sum(-1, keepdim=True)
    out = (w @ v.permute(0, 2, 1, 3).contiguous()) / total.masked_fill(total == 0, 1.0)

    def rows(x):   # [batch][kv][max_q * group][...] -> [tokens][heads][...]
        x = x.view(c["batch"], c["kv"], s["max_q"], group, -1).transpose(1, 2)[seq, row]
        return x.reshape(t.numel(), c["heads"], -1)

    out = rows(out).to(s["q"].dtype)
    return {"out": out, "lse": rows(top + total.log())[..., 0]} if c["lse"] else {"out": out}


def _in_order(outputs):
    return {k: outputs[k] for k in sorted(outputs)}


def run(state):
    s = state
    c = s["c"]
    if not own:
        if c["op"] == "attend":
            return _plain_attend(s)
        out = {} if c["pass_"] == "backward" else _plain_forward(s)
        if c["pass_"] != "forward":
            out.update(_plain_backward(s, s["h"] if "h" in s else out["h"]))
        return _in_order(out)
    if c["op"] == "joint":
        from mamba_ssm_scan_amd import norm
        kw = {k: s[k] for k in ("gate", "scale", "post_weight", "weight") if s[k] is not None}
        if c["gate"]:
            kw["gate_fn"] = c["gate"]
        if c["pass_"] == "backward":
            g = norm.residual_norm_backward(s["dh"], s["dy"], s["h"], s["o"], eps=EPS, **kw)
            return _in_order({"d" + k: v for k, v in g.items() if v is not None})
        if c["pass_"] == "forward":
            got = norm.residual_norm(s["x"], s["o"], eps=EPS, **kw)
            return {"h": got[0], "y": got[1]} if c["pre"] else {"h": got}
        leaf = {k: s[k].detach().requires_grad_() for k in ("x", "o", "gate", "scale", "post_weight", "weight")
                if s[k] is not None}
        h, y = norm.residual_norm(**leaf, eps=EPS, **({"gate_fn": c["gate"]} if c["gate"] else {}))
        grads = torch.autograd.grad([h, y], list(leaf.values()), [s["dh"], s["dy"]])
        return _in_order(dict({"h": h.detach(), "y": y.detach()}, **{"d" + k: g for k, g in zip(leaf, grads)}))
    from mamba_ssm_scan_amd import attention
    if "cache" not in s:
        s["cache"] = attention.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["prefix"] = attention.SharedPrefix(s["shared"], s["count"], s["cu_seqs"]) if c.get("groups") else None
    got = s["cache"].attend(s["q"], s["kv_len"], s["pages"], cu_q=None if s["each_one"] else s["cu_q"], max_q=s["max_q"],
                            max_kv=s["max_kv"], window=c["window"], sinks=c["sinks"], prefix=s["prefix"], lse=c["lse"])
    return {"out": got[0], "lse": got[1]} if c["lse"] else {"out": got}


# ---------------------------------------------------------------------------------------------------------- needs

def work(case):
    c = case
    if c["op"] == "joint":
        n, io, res = c["tokens"] * c["width"], 2 if c["io"] == "bf16" else 4, 2 if c["res"] == "bf16" else 4
        gate, vectors = io * bool(c["gate"]), 4 * c["width"] * (c["post"] + c["scale"] + c["pre"])
        forward = n * (2 * res + io + gate + io * c["pre"]) + vectors
        backward = n * (3 * res + 3 * io + 2 * gate) + 2 * vectors
        if c["pass_"] == "train":   # x, o, gate, dh, dy in; h, y and the gradients out
            return {"bytes": n * (4 * res + 4 * io + 2 * gate) + 2 * vectors, "flops": 50 * n}
        return {"bytes": forward, "flops": 15 * n} if c["pass_"] == "forward" else {"bytes": backward, "flops": 35 * n}
    n, held, cu_seqs, count = _lengths(c)
    size, row = 2 if c["io"] == "bf16" else 4, c["kv"] * c["dim"]
    keys = pairs = 0
    for a, b, k in zip(cu_seqs, cu_seqs[1:], count):
        pre = k * c["page"]
        keys += pre if any(held[i] and n[i] for i in range(a, b)) else 0
        for i in range(a, b):
            if not held[i] or not n[i]:
                continue
            low = max(0, held[i] - n[i] - c["window"] + 1) if c["window"] else 0
            keys += held[i] - max(low, pre) + min(c["sinks"], low)
            for p in range(held[i] - n[i], held[i]):
                low = max(0, p - c["window"] + 1) if c["window"] else 0
                pairs += p + 1 - low + min(c["sinks"], low)
    move = 2 * keys * row + 8 * c["kv"] * (keys // BLOCK) + 2 * sum(n) * c["heads"] * c["dim"] * size
    return {"bytes": move + 4 * sum(n) * c["heads"] * c["lse"], "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---------------------------------------------------------------------------------------------------------- 64 bits

def _exact_joint(s):
    """The definition as a graph in 64 bits; its gradients by automatic differentiation, at the stream as stored."""
    c = s["c"]
    leaf = {k: s[k].double().requires_grad_() for k in ("o", "gate", "scale", "post_weight", "weight") if s[k] is not None}

    def norm(v, w):
        return w * v / (v.square().sum(-1, keepdim=True) / c["width"] + EPS).sqrt()

    with torch.enable_grad():
        b = leaf["o"] if "post_weight" not in leaf else norm(leaf["o"], leaf["post_weight"])
        if c["gate"]:
            g = leaf["gate"]
            b = b * {"identity": g, "sigmoid": torch.sigmoid(g), "silu": g * torch.sigmoid(g)}[c["gate"]]
        b = b * leaf["scale"] if "scale" in leaf else b
        got, h = {}, s.get("h")
        if h is None:
            h = s["x"].double() + b.detach()
            got["h"] = h
            if "weight" in leaf:
                got["y"] = norm(h, leaf["weight"]).detach()
            h = h.to(s["x"].dtype)
        if c["pass_"] == "forward":
            return got
        h = h.double().requires_grad_()
        dh, dw = torch.autograd.grad(norm(h, leaf["weight"]), [h, leaf["weight"]], s["dy"].double())
        got["dx"], got["dweight"] = s["dh"].double() + dh, dw
        rest = [k for k in leaf if k != "weight"]
        for k, g in zip(rest, torch.autograd.grad(b, [leaf[k] for k in rest], got["dx"])):
            got["d" + k] = g
    return got


def _exact_attend(s):
    c = s["c"]
    n, held, cu_seqs, count = _lengths(c)
    group, dev = c["heads"] // c["kv"], s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=dev)
    row = 0
    for i, (k, h) in enumerate(zip(n, held)):
        if k and h:
            g = max(j for j in range(len(count)) if cu_seqs[j] <= i)
            table = s["pages"][i, :-(-h // c["page"])].clone()
            table[:count[g]] = s["shared"][g, :count[g]][:table.numel()]
            pg = table.long().clamp(min=0)
            kk = s["k"].view(torch.int8)[pg].view(s["k"].dtype)
            kk = (kk.double() * s["k_scale"][pg].double()[..., None, None]).transpose(0, 1).reshape(c["kv"], -1, c["dim"])[:, :h]
            vv = s["v"].view(torch.int8)[pg].view(s["v"].dtype)
            vv = (vv.double() * s["v_scale"][pg].double()[..., None, None]).transpose(-1, -2)
            vv = vv.transpose(0, 1).reshape(c["kv"], -1, c["dim"])[:, :h]
            there, place = torch.arange(h, device=dev), torch.arange(h - k, h, device=dev)[:, None]
            hidden = there > place
            if c["window"]:
                hidden = hidden | ((there <= place - c["window"]) & (there >= c["sinks"]))
            for head in range(c["heads"]):
                w = s["q"][row:row + k, head].double() @ kk[head // group].T / math.sqrt(c["dim"])
                w.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(w, -1, keepdim=True)
                lse[row:row + k, head] = z[:, 0]
                out[row:row + k, head] = (w - z).exp().nan_to_num(0.0) @ vv[head // group]
        row += k
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return _in_order(_exact_joint(s)) if case["op"] == "joint" else _exact_attend(s)


if __name__ == "__main__":
    for k in listed() + [draw(random.Random(j)) for j in range(12)]:
        print(k, work(k))
