"""Timed cases of the attention layer's operators: rotary positions, the paged 8-bit cache's append, and attention over it.

A hybrid stack puts one attention layer next to several recurrent mixers; these are that layer's calls. Each case names
its sizes; `prepare` draws its inputs, `run` makes one pass, in plain torch operations in 32 bits or through the
package's kernels (`own`), and `exact` evaluates the definitions in 64 bits.

The cache holds tokens in pages of `page` tokens, each (page, head) as blocks of 16 tokens with one scale a block:
K codes [pages][heads][page / 16][16][dim], V codes [pages][heads][page / 16][dim][16], scales [pages][heads][page / 16];
a value is its code times its block's scale. Sequence i holds its tokens in the pages `pages[i]` names, in order.
"""
import math
import random

import torch

own = False

BLOCK = 16                                   # tokens that share a scale
CODE = {"int8": (torch.int8, 127.0), "fp8": (torch.float8_e4m3fn, 448.0)}
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one step of a batch of 128: the queries of one token each, where only the launch counts
        dict(name="rope_step_b128", op="rope", io="bf16", tokens=128, heads=16, dim=128, rot=128, inter=False,
             first=1, last=4096, back=False),
        # a training batch of 4 sequences of 2048 tokens, all 32 heads
        dict(name="rope_train_4x2048", op="rope", io="bf16", tokens=8192, heads=32, dim=64, rot=64, inter=False,
             first=0, last=2047, back=False),
        # its gradient in 32 bits, neighbouring pairs, half of each head turned, an odd count, late positions
        dict(name="rope_grad_f32_partial", op="rope", io="f32", tokens=3001, heads=9, dim=80, rot=40, inter=True,
             first=30000, last=33000, back=True),
        # one step of a batch of 128 in mid-answer: blocks are partly filled, one new token each
        dict(name="append_step_b128", op="append", fmt="int8", io="bf16", batch=128, q_lo=1, q_hi=1, ctx_lo=1,
             ctx_hi=2047, idle=0, heads=16, kv=4, dim=128, rot=128, inter=False, page=64),
        # four prompts of 2048 tokens into an empty cache
        dict(name="append_prompt_4x2048", op="append", fmt="fp8", io="bf16", batch=4, q_lo=2048, q_hi=2048, ctx_lo=0,
             ctx_hi=0, idle=0, heads=16, kv=4, dim=128, rot=128, inter=False, page=64),
        # a mixed batch: pieces of prompts and single tokens at any place of a block, idle slots, small pages
        dict(name="append_mixed_f32", op="append", fmt="int8", io="f32", batch=13, q_lo=0, q_hi=77, ctx_lo=0,
             ctx_hi=1001, idle=2, heads=6, kv=3, dim=80, rot=40, inter=True, page=16),
        # one conversation, one token: the smallest call
        dict(name="attend_one_ctx2048", op="attend", fmt="int8", io="bf16", batch=1, q_lo=1, q_hi=1, ctx_lo=2047,
             ctx_hi=2047, idle=0, heads=16, kv=4, dim=128, page=64, window=0, causal=True, lse=False),
        # a serving batch of 128 at many lengths, some slots idle
        dict(name="attend_step_b128", op="attend", fmt="int8", io="bf16", batch=128, q_lo=1, q_hi=1, ctx_lo=127,
             ctx_hi=4095, idle=3, heads=16, kv=4, dim=128, page=64, window=0, causal=True, lse=True),
        # a few conversations over very long contexts
        dict(name="attend_step_b4_ctx131071", op="attend", fmt="fp8", io="bf16", batch=4, q_lo=1, q_hi=1,
             ctx_lo=131071, ctx_hi=131071, idle=0, heads=32, kv=4, dim=128, page=64, window=0, causal=True, lse=False),
        # four prompts of 2048 tokens
        dict(name="attend_prompt_4x2048", op="attend", fmt="int8", io="bf16", batch=4, q_lo=2048, q_hi=2048, ctx_lo=0,
             ctx_hi=0, idle=0, heads=32, kv=8, dim=64, page=64, window=0, causal=True, lse=False),
        # the last piece of a prompt of 32768 tokens
        dict(name="attend_piece_2048_of_32768", op="attend", fmt="fp8", io="bf16", batch=1, q_lo=2048, q_hi=2048,
             ctx_lo=30720, ctx_hi=30720, idle=0, heads=16, kv=4, dim=128, page=64, window=0, causal=True, lse=False),
        # 32-bit checks of a model with a sliding window: drafts of a few tokens, odd lengths, small pages
        dict(name="attend_draft_f32_window", op="attend", fmt="int8", io="f32", batch=7, q_lo=0, q_hi=5, ctx_lo=0,
             ctx_hi=3001, idle=1, heads=6, kv=3, dim=80, page=16, window=511, causal=True, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    io = rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    rot = rng.choice([dim, dim, dim // 2, 16])
    inter = rng.random() < 0.4
    if op == "rope":
        heads, cap = _log(rng, 1, 64), (1 << 24) if io == "bf16" else (1 << 23)
        first = _log(rng, 1, 500000) - 1
        tokens = min(_log(rng, 1, 9000), cap // (heads * dim))
        return dict(op=op, io=io, tokens=tokens, heads=heads, dim=dim, rot=rot, inter=inter, first=first,
                    last=first + _log(rng, 1, 9000), back=rng.random() < 0.4)
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 6, 8, 16])
    fmt = rng.choice(["int8", "fp8"])
    page = rng.choice([16, 32, 64, 128, 256])
    idle = rng.choice([0, 0, 1])
    if op == "append":
        q_hi = min(rng.choice([1, _log(rng, 1, 2048)]), max(1, (1 << 23) // (heads * dim)))
        batch = min(_log(rng, 1, 130), max(1, (1 << 23) // (q_hi * heads * dim)), 2 + 8192 // (q_hi + 64))
        q_lo = rng.choice([0, q_hi, max(0, q_hi // 3)]) if q_hi > 1 else 1
        ctx_hi = _log(rng, 1, 3000) - 1
        return dict(op=op, fmt=fmt, io=io, batch=batch, q_lo=q_lo, q_hi=q_hi, ctx_lo=rng.choice([0, ctx_hi // 2]),
                    ctx_hi=ctx_hi, idle=min(idle, batch - 1), heads=heads, kv=kv, dim=dim, rot=rot, inter=inter,
                    page=page)
    kind = rng.choice(["step", "step", "draft", "prompt", "piece"])
    causal, window = True, 0
    if kind in ("step", "draft"):
        q_hi = 1 if kind == "step" else rng.randint(2, 9)
        ctx_hi = _log(rng, 1, 130000)
        batch = max(1, min(_log(rng, 1, 130), (1 << 28) // ((ctx_hi + q_hi + page) * kv * dim),
                           (1 << 29) // (ctx_hi * heads * q_hi)))
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
    else:
        q_hi = min(_log(rng, 10, 2048), int(math.sqrt((1 << 28) / heads)))
        ctx_hi = 0 if kind == "prompt" else min(_log(rng, 1, 30000), (1 << 28) // (q_hi * heads) + 1)
        batch = max(1, min(_log(rng, 1, 8), (1 << 28) // ((ctx_hi + q_hi) * q_hi * heads)))
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        causal = window > 0 or rng.random() < 0.8
    return dict(op=op, fmt=fmt, io=io, batch=batch, q_lo=rng.choice([q_hi, q_hi, max(0, q_hi // 2)]) if q_hi > 1 else 1,
                q_hi=q_hi, ctx_lo=rng.choice([ctx_hi, ctx_hi // 3]), ctx_hi=ctx_hi, idle=min(idle, batch - 1),
                heads=heads, kv=kv, dim=dim, page=page, window=window, causal=causal, lse=rng.random() < 0.3)


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi (the first is hi), spread by the multiples of an irrational number."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * (((i + 1) * step) % 1.0)) for i in range(n)]


def _lengths(c):
    """(new tokens, tokens held after the call) of each sequence; idle slots hold none and still bring a query row."""
    n = _spread(c["q_lo"], c["q_hi"], c["batch"], 0.7548776662466927)
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["batch"], 0.6180339887498949)
    held = [a + b for a, b in zip(n, ctx)]
    for i in range(c["idle"]):
        held[c["batch"] - 1 - i] = 0
    return n, held


# ---------------------------------------------------------------------------------------------------------- inputs

def _frequencies(rot):
    return torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float32)


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
    io = IO[c["io"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(io)

    if c["op"] == "rope":
        positions = c["first"] + torch.arange(c["tokens"], device=dev) % (c["last"] - c["first"] + 1)
        positions = positions[torch.randperm(c["tokens"], generator=gen, device=dev)].to(torch.int32)
        return dict(c=c, x=normal(c["tokens"], c["heads"], c["dim"]), positions=positions,
                    freq=_frequencies(c["rot"]).to(dev))
    n, held = _lengths(c)
    max_pages = max(1, max(-(-h // c["page"]) for h in held))
    need = [-(-h // c["page"]) for h in held]
    num_pages = sum(need) + 3
    order = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    pages = torch.zeros((c["batch"], max_pages), dtype=torch.int32, device=dev)
    at = 0
    for i, k in enumerate(need):
        pages[i, :k] = order[at:at + k]
        at += k
    cu = [0]
    for k in n:
        cu.append(cu[-1] + k)
    tokens = cu[-1]
    s = dict(c=c, pages=pages, kv_len=torch.tensor(held, dtype=torch.int32, device=dev),
             cu_q=torch.tensor(cu, dtype=torch.int32, device=dev), max_q=max(1, max(n)), max_kv=max(1, max(held)),
             q=normal(tokens, c["heads"], c["dim"]), **_fill_pool(c, num_pages, gen, dev))
    s["each_one"] = n == [1] * c["batch"]
    if c["op"] == "append":
        begun = [max(0, h - k) // BLOCK * BLOCK for k, h in zip(n, held)]   # of the first block that the call touches
        s["first"] = torch.tensor(begun, dtype=torch.int32, device=dev)
        s["count"] = torch.tensor([h - f if k else 0 for k, h, f in zip(n, held, begun)], dtype=torch.int32, device=dev)
        s["max_count"] = max(1, max(h - f if k else 0 for k, h, f in zip(n, held, begun)))
        s["k_new"] = 2.0 * normal(tokens, c["kv"], c["dim"])
        s["v_new"] = normal(tokens, c["kv"], c["dim"])
        s["freq"] = _frequencies(c["rot"]).to(dev)
        touched = [(i, j) for i, (k, h, f) in enumerate(zip(n, held, begun)) if k for j in range(-(-(h - f) // BLOCK))]
        s["touched"] = torch.tensor(touched, dtype=torch.int64, device=dev).view(-1, 2)   # (sequence, block of the call)
        kept = [r for i, (k, h) in enumerate(zip(n, held)) if h for r in range(cu[i], cu[i] + k)]
        s["kept"] = torch.tensor(kept, dtype=torch.int64, device=dev)                    # rows of live slots
    return s


# ---------------------------------------------------------------------------------------------------------- plain forms

def _turn(x, positions, freq, inter, sign):
    """Rows of x [tokens][heads][dim] turned by their positions' angles (formed in 64 bits, as a position may be large)."""
    rot = 2 * freq.numel()
    angle = positions.double()[:, None] * freq.double()
    cos, sin = angle.cos().float()[:, None, :], sign * angle.sin().float()[:, None, :]
    y = x.float().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    xa, xb = x[..., a].float(), x[..., b].float()
    y[..., a] = xa * cos - xb * sin
    y[..., b] = xa * sin + xb * cos
    return y


def _sequence_of(s):
    """(sequence, position) of each row."""
    t = torch.arange(s["q"].shape[0], device=s["q"].device)
    seq = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    return seq, s["kv_len"].long()[seq] - n[seq] + t - s["cu_q"].long()[seq]


def _dense(s, pos, seq):
    """The values the cache holds at positions pos of sequences seq (both of one shape), [...][heads][dim] in 32 bits."""
    page = s["c"]["page"]
    pg = s["pages"].long()[seq, (pos // page).clamp(max=s["pages"].shape[1] - 1)]
    sub, slot = pos % page // BLOCK, pos % BLOCK
    k = s["k"].view(torch.int8)[pg, :, sub, slot].view(s["k"].dtype).float() * s["k_scale"][pg, :, sub][..., None]
    v = s["v"].view(torch.int8)[pg, :, sub, :, slot].view(s["v"].dtype).float() * s["v_scale"][pg, :, sub][..., None]
    return k, v


def _plain_append(s):
    c = s["c"]
    dt, top = CODE[c["fmt"]]
    seq, pos = _sequence_of(s)
    q = _turn(s["q"], pos, s["freq"], c["inter"], 1.0).to(s["q"].dtype)
    new = {"k": _turn(s["k_new"], pos, s["freq"], c["inter"], 1.0), "v": s["v_new"].float()}
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    before = s["kv_len"].long() - n
    begun = before.clamp(min=0) // BLOCK
    blocks = (s["max_q"] + BLOCK - 2) // BLOCK + 1
    b = torch.arange(c["batch"], device=pos.device)[:, None]
    blk = begun[:, None] + torch.arange(blocks, device=pos.device)
    at = blk[..., None] * BLOCK + torch.arange(BLOCK, device=pos.device)               # position of each slot
    fresh = (at >= before[:, None, None]) & (at < s["kv_len"].long()[:, None, None])
    old = at < before[:, None, None]
    per = c["page"] // BLOCK
    pg = s["pages"].long()[b, (blk // per).clamp(max=s["pages"].shape[1] - 1)]
    kept, (i, j) = s["kept"], s["touched"].unbind(1)
    page, sub = pg[i, j], (blk % per)[i, j]
    for name in ("k", "v"):
        buf = torch.zeros((c["batch"], blocks, BLOCK, c["kv"], c["dim"]), device=pos.device)
        buf[seq[kept], pos[kept] // BLOCK - begun[seq[kept]], pos[kept] % BLOCK] = new[name][kept]
        buf = buf.permute(0, 1, 3, 2, 4)                                                # [batch][block][head][slot][dim]
        held = s[name].view(torch.int8)[pg, :, blk % per].view(dt).float()
        held = held if name == "k" else held.transpose(-1, -2)
        had = torch.where(old.any(-1)[..., None], s[name + "_scale"][pg, :, blk % per], 0.0)
        scale = torch.maximum(had, buf.abs().amax((-1, -2)) / top)
        inv = torch.where(scale > 0, 1.0 / scale, 0.0)
        y = torch.where(old[:, :, None, :, None], held * (had * inv)[..., None, None], 0.0)
        y = torch.where(fresh[:, :, None, :, None], buf * inv[..., None, None], y)
        y = (y.round() if c["fmt"] == "int8" else y).clamp(-top, top).to(dt)
        y = y if name == "k" else y.transpose(-1, -2)
        s[name].view(torch.int8)[page, :, sub] = y.contiguous().view(torch.int8)[i, j]
        s[name + "_scale"][page, :, sub] = scale[i, j]
    at = s["first"].long()[:, None] + torch.arange(s["max_count"], device=pos.device)
    there = torch.arange(s["max_count"], device=pos.device) < s["count"][:, None]
    k, v = _dense(s, at, b.expand_as(at))
    k, v = (torch.where(there[..., None, None], x, 0.0).to(s["q"].dtype) for x in (k, v))
    return {"q": q, "k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_attend(s):
    c = s["c"]
    seq, pos = _sequence_of(s)
    dev, group = pos.device, c["heads"] // c["kv"]
    row = torch.arange(pos.numel(), device=dev) - s["cu_q"].long()[seq]
    q = torch.zeros((c["batch"], s["max_q"], c["kv"], group, c["dim"]), device=dev)
    q[seq, row] = s["q"].float().view(-1, c["kv"], group, c["dim"]) / math.sqrt(c["dim"])
    at = torch.arange(s["max_kv"], device=dev).expand(c["batch"], -1)
    k, v = _dense(s, at, torch.arange(c["batch"], device=dev)[:, None].expand_as(at))
    place = torch.full((c["batch"], s["max_q"]), -1, device=dev)
    place[seq, row] = pos
    seen = at[:, None, :] < s["kv_len"].long()[:, None, None]
    seen = seen.expand(-1, s["max_q"], -1)
    if c["causal"]:
        seen = seen & (at[:, None, :] <= place[..., None])
    if c["window"]:
        seen = seen & (at[:, None, :] > place[..., None] - c["window"])
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, group, -1).reshape(c["batch"], 1, -1, s["max_kv"])
    w = q.permute(0, 2, 1, 3, 4).reshape(c["batch"], c["kv"], -1, c["dim"]) @ k.permute(0, 2, 3, 1)
    w = w.masked_fill(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = (w - top.clamp(min=-3.0e38)).exp()
    total = w.sum(-1, keepdim=True)
    out = (w @ v.permute(0, 2, 1, 3)) / total.masked_fill(total == 0, 1.0)

    def rows(x):   # [batch][kv][max_q * group][...] -> [tokens][heads][...]
        x = x.view(c["batch"], c["kv"], s["max_q"], group, -1).transpose(1, 2)[seq, row]
        return x.reshape(pos.numel(), c["heads"], -1)

    out = rows(out).to(s["q"].dtype)
    return {"out": out, "lse": rows(top + total.log())[..., 0]} if c["lse"] else {"out": out}


def run(state):
    s = state
    c = s["c"]
    if not own:
        if c["op"] == "rope":
            return _turn(s["x"], s["positions"], s["freq"], c["inter"], -1.0 if c["back"] else 1.0).to(s["x"].dtype)
        return _plain_append(s) if c["op"] == "append" else _plain_attend(s)
    from mamba_ssm_scan_amd import attention
    if c["op"] == "rope":
        return attention.rope(s["x"], s["positions"], s["freq"], interleaved=c["inter"], backward=c["back"])
    if "cache" not in s:
        s["cache"] = attention.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    cache, cu = s["cache"], None if s["each_one"] else s["cu_q"]
    if c["op"] == "append":
        q = cache.append(s["k_new"], s["v_new"], s["kv_len"], s["pages"], cu_q=cu, max_q=s["max_q"], q=s["q"],
                         inv_freq=s["freq"], interleaved=c["inter"])
        k, v = cache.read(s["first"], s["count"], s["pages"], s["max_count"], dtype=s["q"].dtype)
        return {"q": q, "k": k, "v": v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    got = cache.attend(s["q"], s["kv_len"], s["pages"], cu_q=cu, max_q=s["max_q"], max_kv=s["max_kv"],
                       causal=c["causal"], window=c["window"], lse=c["lse"])
    return {"out": got[0], "lse": got[1]} if c["lse"] else {"out": got}


# ---------------------------------------------------------------------------------------------------------- needs

def work(case):
    c = case
    size = 2 if c["io"] == "bf16" else 4
    if c["op"] == "rope":
        return {"bytes": c["tokens"] * (2 * c["heads"] * c["dim"] * size + 4), "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    n, held = _lengths(c)
    tokens, row = sum(n), c["kv"] * c["dim"]
    if c["op"] == "append":
        new = sum(min(k, h) for k, h in zip(n, held))
        old = sum((h - k) % BLOCK for k, h in zip(n, held) if 0 < k <= h)
        blocks = sum((h - 1) // BLOCK - (h - k) // BLOCK + 1 for k, h in zip(n, held) if 0 < k <= h)
        move = tokens * 2 * c["heads"] * c["dim"] * size        # q in and out
        move += 2 * new * row * size                            # K and V in
        move += 2 * (old + blocks * BLOCK) * row + 16 * blocks * c["kv"]    # the codes and scales
        most = max((h - (h - k) // BLOCK * BLOCK for k, h in zip(n, held) if 0 < k <= h), default=1)
        move += 2 * (old + new + c["batch"] * most * size) * row            # and their values, rows of one length
        return {"bytes": move, "flops": 6 * tokens * c["heads"] * c["dim"]}
    keys = pairs = 0
    for k, h in zip(n, held):
        low = max(0, h - k - c["window"] + 1) if c["window"] else 0
        keys += max(0, h - low) if k else 0
        for p in range(h - k, h):
            top = p + 1 if c["causal"] else h
            pairs += max(0, min(top, c["window"]) if c["window"] else top)
    move = 2 * keys * row + 8 * c["kv"] * (keys // BLOCK) + 2 * tokens * c["heads"] * c["dim"] * size
    return {"bytes": move + 4 * tokens * c["heads"] * c["lse"], "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---------------------------------------------------------------------------------------------------------- 64 bits

def _complex_turn(x, positions, freq, inter, sign):
    """The rotation as a product of complex numbers."""
    half = freq.numel()
    head, tail = x.double()[..., :2 * half], x.double()[..., 2 * half:]
    pair = head.unflatten(-1, (half, 2)) if inter else head.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_complex(pair.contiguous())
    phase = positions.double()[:, None, None] * freq.double()
    out = torch.view_as_real(z * torch.polar(torch.ones_like(phase), sign * phase))
    out = out.flatten(-2) if inter else out.transpose(-1, -2).flatten(-2)
    return torch.cat([out, tail], -1)


def _nearest_code(x, fmt):
    """The nearest value that a code stands for, ties to even."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].double() - 4)
    return ((x / step).round() * step).clamp(-448, 448)


def _blocks_of(s, i, name, blks):
    """Blocks `blks` of sequence i as (codes, scales): [block][head][slot][dim], [block][head], in 64 bits."""
    per = s["c"]["page"] // BLOCK
    codes, scales = [], []
    for j in blks:
        p = int(s["host_pages"][i][j // per])
        x = s[name][p, :, j % per].double()
        codes.append(x if name == "k" else x.transpose(-1, -2))
        scales.append(s[name + "_scale"][p, :, j % per].double())
    return torch.stack(codes), torch.stack(scales)


def _exact_append(s):
    c = s["c"]
    top = CODE[c["fmt"]][1]
    n, held = _lengths(c)
    per = c["page"] // BLOCK
    s["host_pages"] = s["pages"].tolist()
    shape = (c["batch"], s["max_count"], c["kv"], c["dim"])
    dev = s["q"].device
    got = {"k": torch.zeros(shape, dtype=torch.float64, device=dev), "v": torch.zeros(shape, dtype=torch.float64, device=dev),
           "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
    pos = torch.cat([torch.arange(h - k, h, device=dev) for k, h in zip(n, held)])
    got["q"] = _complex_turn(s["q"], pos, s["freq"], c["inter"], 1.0)
    new = {"k": _complex_turn(s["k_new"], pos, s["freq"], c["inter"], 1.0), "v": s["v_new"].double()}
    row = 0
    for i, (k, h) in enumerate(zip(n, held)):
        if 0 < k <= h:
            first, last = (h - k) // BLOCK, (h - 1) // BLOCK
            skip = (h - k) % BLOCK
            for name in ("k", "v"):
                rows = new[name][row:row + k]
                room = torch.zeros(((last - first + 1) * BLOCK, c["kv"], c["dim"]), dtype=torch.float64, device=dev)
                room[skip:skip + k] = rows
                room = room.view(-1, BLOCK, c["kv"], c["dim"]).transpose(1, 2).clone()
                scale = room.abs().amax((-1, -2)) / top
                if skip:
                    codes, scales = _blocks_of(s, i, name, [first])
                    scale[0] = torch.maximum(scale[0], scales[0])
                unit = torch.where(scale > 0, scale, torch.ones_like(scale))[..., None, None]
                room = _nearest_code(room / unit, c["fmt"]) * unit
                if skip:
                    kept = _nearest_code(codes[0] * (scales[0][:, None, None] / unit[0]), c["fmt"]) * unit[0]
                    room[0, :, :skip] = kept[:, :skip]
                got[name][i, :skip + k] = room.transpose(1, 2).reshape(-1, c["kv"], c["dim"])[:skip + k]
                for j in range(first, last + 1):
                    got[name + "_scale"][s["host_pages"][i][j // per], :, j % per] = scale[j - first]
        row += k
    return got


def _exact_attend(s):
    c = s["c"]
    n, held = _lengths(c)
    s["host_pages"] = s["pages"].tolist()
    group, dev = c["heads"] // c["kv"], s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=dev)
    row = 0
    for i, (k, h) in enumerate(zip(n, held)):
        if k and h:
            pg = s["pages"][i, :-(-h // c["page"])].long()
            kk = s["k"].view(torch.int8)[pg].view(s["k"].dtype)
            kk = (kk.double() * s["k_scale"][pg].double()[..., None, None]).transpose(0, 1).reshape(c["kv"], -1, c["dim"])[:, :h]
            vv = s["v"].view(torch.int8)[pg].view(s["v"].dtype)
            vv = (vv.double() * s["v_scale"][pg].double()[..., None, None]).transpose(-1, -2)
            vv = vv.transpose(0, 1).reshape(c["kv"], -1, c["dim"])[:, :h]
            there, place = torch.arange(h, device=dev), torch.arange(h - k, h, device=dev)[:, None]
            hidden = torch.zeros((k, h), dtype=torch.bool, device=dev)
            if c["causal"]:
                hidden |= there > place
            if c["window"]:
                hidden |= there <= place - c["window"]
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
    if case["op"] == "rope":
        return _complex_turn(s["x"], s["positions"], s["freq"], case["inter"], -1.0 if case["back"] else 1.0)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


if __name__ == "__main__":
    for k in listed() + [draw(random.Random(j)) for j in range(8)]:
        print(k, work(k))
