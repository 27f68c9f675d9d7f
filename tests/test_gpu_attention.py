"""Rotary positions, the paged 8-bit cache and attention over it (mamba_ssm_scan_amd.attention) against 64-bit definitions."""
import math

import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu

BF, F32, I8, F8 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
DEV = "cuda"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g).to(dtype)


def within(got, want, bound, what=""):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, what
    bad = (got - want).abs() > bound
    bad |= torch.isnan(got) != torch.isnan(want)
    worst = ((got - want).abs() / bound).nan_to_num(0.0).max().item() if got.numel() else 0.0
    print(f"  {what}: largest error / bound {worst:.3f}", flush=True)
    assert not bad.any(), f"{what}: {int(bad.sum())} entries off, largest error / bound {worst:.3g}"


def turn_bound(x, y, mscale, dtype):
    """Two products and a sum in fp32 (3 roundings of at most the pair's magnitude), (cos, sin) rounded to fp32, and
    the io rounding of the result."""
    mag = x.double().abs().amax(-1, keepdim=True) * 2 * max(1.0, abs(mscale))
    return mag * 2.0 ** -22 + y.abs() * (2.0 ** -8 if dtype == BF else 2.0 ** -24) + 1e-30


# ---------------------------------------------------------------------------------------------------------- rope

ROPE = [  # tokens, heads, dim, rot, interleaved, dtype, mscale
    (1, 1, 64, 64, False, BF, 1.0), (7, 3, 128, 128, False, F32, 1.0), (5, 4, 64, 32, True, BF, 1.3),
    (300, 2, 80, 40, True, F32, 1.0), (33, 5, 96, 48, False, F32, 0.7), (9, 2, 20, 6, False, BF, 1.0),
    (3, 1, 2, 2, True, F32, 1.0), (17, 3, 30, 10, True, F32, 1.0), (2100, 4, 32, 16, False, BF, 1.0),
    (4, 2, 4096, 4096, False, F32, 1.0), (2, 1, 2500, 2406, True, BF, 1.0), (0, 3, 64, 64, False, BF, 1.0),
]


@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("case", ROPE, ids=str)
def test_rope(case, backward):
    T, H, D, rot, inter, dt, ms = case
    g = gen(T + D)
    x = normal(g, T, H, D, dtype=dt)
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    f, _ = attention.rope_frequencies(rot, device="cpu")
    y = attention.rope(x.to(DEV), pos.to(DEV), f.to(DEV), interleaved=inter, mscale=ms, backward=backward)
    want = ref.turn(x, pos, f, inter, ms, backward)
    within(y, want, turn_bound(x, want, ms, dt), "rope")


def test_rope_far_and_negative_positions():
    """Angles of late positions keep their fraction of a turn: fp32 angles would be off by whole radians."""
    g = gen(3)
    pos = torch.tensor([-1, -70000, 10 ** 6, 123456789, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    x = normal(g, 6, 2, 64)
    f, _ = attention.rope_frequencies(64, device="cpu")
    y = attention.rope(x.to(DEV), pos.to(DEV), f.to(DEV))
    want = ref.turn(x, pos, f)
    # theta itself has 55 bits and is rounded to 53 once on either side
    within(y, want, turn_bound(x, want, 1.0, F32) + x.double().abs().amax() * 2 * 2.0 ** 31 * 2.0 ** -52, "rope")


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_rope_strides_and_in_place(dt, shift):
    """Heads of a fused projection where they lie, with and without 16-byte alignment; then in place."""
    g = gen(5 + shift)
    T, H, D = 19, 3, 64
    buf = normal(g, T, 5 * D * H + 8, dtype=dt).to(DEV)
    part = buf[:, 8 + shift:8 + shift + H * 2 * D].view(T, H, 2 * D)[:, :, :D]
    pos = torch.arange(T, dtype=torch.int32)
    f, _ = attention.rope_frequencies(D, device="cpu")
    want = ref.turn(part.cpu(), pos, f)
    bound = turn_bound(part.cpu(), want, 1.0, dt)
    before = buf.clone()
    within(attention.rope(part, pos.to(DEV), f.to(DEV)), want, bound, "strided")
    assert torch.equal(buf, before)
    turned = part.transpose(0, 1).contiguous().transpose(0, 1)     # heads outermost
    within(attention.rope(turned, pos.to(DEV), f.to(DEV)), want, bound, "heads outermost")
    assert attention.rope(part, pos.to(DEV), f.to(DEV), out=part) is part
    within(part, want, bound, "in place")
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[:, 8 + shift:8 + shift + H * 2 * D].view(T, H, 2 * D)[:, :, :D] = False
    assert torch.equal(buf[mask], before[mask])                    # the neighbours keep their bits


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(inter):
    """The backward map against differences of a loss, and <R x, dy> = <x, R^T dy>."""
    g = gen(9)
    T, H, D, rot, ms = 6, 2, 24, 16, 1.25
    x, dy, u = (normal(g, T, H, D).to(DEV) for _ in range(3))
    pos = torch.randint(0, 900, (T,), generator=g, dtype=torch.int32).to(DEV)
    f, _ = attention.rope_frequencies(rot)
    kw = dict(interleaved=inter, mscale=ms)
    dx = attention.rope(dy, pos, f, backward=True, **kw).double()
    loss = lambda z: (attention.rope(z, pos, f, **kw).double() * dy.double()).sum()  # noqa: E731
    # the map is linear: a difference has no truncation error, only fp32 rounding of about T H D terms
    diff = (loss(x + u) - loss(x - u)) / 2
    assert abs(float(diff - (dx * u.double()).sum())) <= 2.0 ** -21 * T * H * D * 16
    assert abs(float(loss(x) - (dx * x.double()).sum())) <= 2.0 ** -21 * T * H * D * 16


def test_rope_frequencies():
    f, m = attention.rope_frequencies(64, device="cpu")
    assert m == 1.0 and torch.allclose(f.double(), 10000.0 ** (-torch.arange(32).double() / 32), rtol=1e-6)
    g, _ = attention.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(g, f / 4, rtol=1e-6)
    g, _ = attention.rope_frequencies(64, scaling="base", factor=8.0, device="cpu")
    assert g[0] == f[0] and abs(float(f[-1] / g[-1]) - 8.0) < 1e-4
    g, m = attention.rope_frequencies(64, scaling="bands", factor=4.0, trained_len=2048, device="cpu")
    assert torch.equal(g[:4], f[:4]) and torch.allclose(g[-4:], f[-4:] / 4, rtol=1e-6) and m == 0.1 * math.log(4) + 1
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, scaling="x"), dict(rot=8, scaling="linear", factor=0.5),
                dict(rot=8, scaling="bands", factor=2.0)):
        with pytest.raises(ValueError):
            attention.rope_frequencies(device="cpu", **bad)


# ---------------------------------------------------------------------------------------------------------- cache

class Bench:
    """A cache on the device and its 64-bit counterpart, appended to side by side."""

    def __init__(self, batch, heads, dim, page, room, fmt, seed=0, spare=2):
        g = gen(100 + seed)
        self.g, self.batch, self.heads, self.dim, self.page, self.fmt = g, batch, heads, dim, page, fmt
        per = -(-room // page)
        self.n_pages = batch * per + spare
        self.cache = attention.KVCache.empty(self.n_pages, page, heads, dim, dtype=fmt)
        # memory as it may be found: every byte pattern, the format's NaN among them; scales NaN
        for t in (self.cache.k, self.cache.v):
            t.view(I8).copy_(torch.randint(-128, 128, t.shape, generator=g, dtype=I8))
            t.view(I8)[..., ::3] = 0x7F
        self.cache.k_scale.fill_(float("nan"))
        self.cache.v_scale.fill_(float("nan"))
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.pages = order[:batch * per].view(batch, per).to(DEV)
        self.spare = order[batch * per:].long()
        self.ref = ref.Cache(batch, heads, dim, per * page, fmt)
        self.len = [0] * batch

    def append(self, n, q_heads=0, inv_freq=None, inter=False, mscale=1.0, io=F32, loud=1.0, rows=None):
        T = sum(n)
        k, v = rows if rows else (loud * normal(self.g, T, self.heads, self.dim, dtype=io),
                                  normal(self.g, T, self.heads, self.dim, dtype=io))
        q = normal(self.g, T, q_heads, self.dim, dtype=io) if q_heads else None
        pos = torch.cat([torch.arange(l, l + c) for l, c in zip(self.len, n)]) if T else torch.zeros(0)
        kt = k if inv_freq is None else ref.turn(k, pos, inv_freq, inter, mscale).float()
        at = 0
        for i, c in enumerate(n):
            self.ref.append(i, self.len[i], kt[at:at + c], v[at:at + c])
            self.len[i] += c
            at += c
        cu = None if n == [1] * self.batch else torch.tensor([sum(n[:j]) for j in range(len(n) + 1)],
                                                             dtype=torch.int32, device=DEV)
        out = self.cache.append(k.to(DEV), v.to(DEV), self.kv_len(), self.pages, cu_q=cu, max_q=max(n + [1]),
                                q=None if q is None else q.to(DEV), inv_freq=None if inv_freq is None else inv_freq.to(DEV),
                                interleaved=inter, mscale=mscale)
        if q is not None:
            want = q.double() if inv_freq is None else ref.turn(q, pos, inv_freq, inter, mscale)
            within(out, want, turn_bound(q, want, mscale, io), "q")
        return cu

    def kv_len(self):
        return torch.tensor(self.len, dtype=torch.int32, device=DEV)

    def held(self, dtype=F32):
        top = max(self.len + [1])
        zero = torch.zeros(self.batch, dtype=torch.int32, device=DEV)
        return self.cache.read(zero, self.kv_len(), self.pages, top, dtype=dtype)

    def check(self, times=1, rare=True):
        """Every value held is the definition's, or the neighbouring code where the value lay between the two: a
        rotation and a division in fp32 move x / scale by less than 2^-20 of the range, so the quotient may fall on
        the other side of a tie. `times`: requantisations, each of which may add such a step. Ties are rare (and then
        counted) where values are spread finely; bf16 rows, 8 bits like the codes, meet them whenever the block's
        maximum is a simple multiple of the others."""
        got = self.held()
        for name, x, want, sc in (("k", got[0], self.ref.k, self.ref.ks), ("v", got[1], self.ref.v, self.ref.vs)):
            for i, l in enumerate(self.len):
                w, s = want[i, :l], sc[i].repeat_interleave(16, 0)[:l, :, None]
                g = x[i, :l].cpu().double()
                u = torch.where(s > 0, s, torch.ones_like(s))
                step = ref.step_of(w / u, self.fmt) * s
                assert ((g - w).abs() <= (2.0 ** -20 * self.ref.top) * s + times * step * 1.0001).all(), (name, i)
                off = ((g - w).abs() > 2.0 ** -20 * self.ref.top * s + 1e-30).double().mean().item() if l else 0.0
                assert not rare or off <= 1e-3 * times + 2.0 / max(1, w.numel()), (name, i, off)
                assert (x[i, l:] == 0).all()

    def attend(self, q, n, io, causal=True, window=0, scale=None, max_kv=None, max_q=None, cu=None, lens=None, lse=True,
               gone=(), **kw):
        """The cache's attention against the 64-bit one over the values it holds."""
        lens = lens if lens is not None else self.len
        kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
        pages = self.pages.clone()
        for i, p in gone:
            pages[i, p] = -1
        if cu is None and n != [1] * self.batch:
            cu = torch.tensor([sum(n[:j]) for j in range(len(n) + 1)], dtype=torch.int32, device=DEV)
        got = self.cache.attend(q.to(DEV) if not q.is_cuda else q, kv_len, pages, cu_q=cu,
                                max_q=max(n + [1]) if max_q is None else max_q, max_kv=max_kv, scale=scale, causal=causal,
                                window=window, lse=lse, **kw)
        out, l = got if lse else (got, None)
        kd, vd = self.held()
        at = 0
        for i, c in enumerate(n):
            seen = torch.ones(lens[i], dtype=torch.bool)
            for s, p in gone:
                if s == i:
                    seen[p * self.page:(p + 1) * self.page] = False
            qi = q[at:at + c].cpu()
            o, z, mag, top = ref.attend(qi, torch.arange(lens[i] - c, lens[i]), kd[i, :lens[i]].cpu(), vd[i, :lens[i]].cpu(),
                                        1 / math.sqrt(self.dim) if scale is None else scale, causal, window, seen)
            within(out[at:at + c], o, ref.attend_bound(o, mag, top, self.dim, lens[i], io), f"out {i}")
            if lse:
                zb = 2.0 ** -24 * (lens[i] + (self.dim + 4) * top + 8) * 2 + z.abs() * 2.0 ** -22 + 1e-6
                g = l[at:at + c].cpu().double()
                assert torch.equal(torch.isinf(g), torch.isinf(z)) and (((g - z).abs() <= zb) | torch.isinf(z)).all()
            at += c
        return out


APPEND = [  # batch, heads, dim, page, fmt, io, rot, interleaved, steps of new tokens per sequence
    (1, 1, 64, 16, I8, BF, 64, False, [[1]] * 20),
    (3, 2, 128, 64, F8, F32, 128, False, [[5, 0, 17], [1, 1, 1], [40, 3, 0], [1, 1, 1]]),
    (2, 3, 80, 32, I8, F32, 40, True, [[0, 33], [16, 16], [1, 1], [70, 15], [1, 1]]),
    (4, 1, 256, 128, F8, BF, 64, False, [[1, 2, 3, 4], [130, 0, 0, 1], [1, 1, 1, 1]]),
    (2, 2, 16, 16, I8, F32, 2, True, [[31, 32], [1, 1], [2, 0]]),
    (2, 4, 192, 16, I8, BF, 0, False, [[7, 100], [9, 1], [1, 1]]),
    (2, 2, 96, 64, F8, F32, 22, False, [[50, 64], [14, 1]]),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(v) for v in c[:8]))
def test_append(case):
    b, H, D, page, fmt, io, rot, inter, steps = case
    bench = Bench(b, H, D, page, 256, fmt, seed=D)
    f = attention.rope_frequencies(rot, device="cpu")[0] if rot else None
    spare_k = bench.cache.k.view(I8)[bench.spare].clone()
    for j, n in enumerate(steps):
        # louder and quieter tokens: the scale grows at some steps and stays at others
        bench.append(n, q_heads=H * (j % 3), inv_freq=f, inter=inter, io=io, loud=[1.0, 4.0, 0.1][j % 3])
        bench.check(times=1 + j, rare=io == F32)
    assert torch.equal(bench.cache.k.view(I8)[bench.spare], spare_k)


def test_append_codes_are_the_formulas():
    """Codes and scales bit for bit, without a rotation: fp32 operations as the header writes them."""
    for fmt, top in ((I8, 127.0), (F8, 448.0)):
        bench = Bench(1, 2, 32, 16, 32, fmt)
        a = normal(bench.g, 5, 2, 32)
        b = 8.0 * normal(bench.g, 4, 2, 32)
        bench.append([5], rows=(a, a))
        p = int(bench.pages[0, 0])
        s = a.abs().amax((0, 2)) * torch.tensor(1.0 / top, dtype=F32)

        def code(x):
            return (x.round() if fmt == I8 else x).clamp(-top, top).to(fmt).view(I8)

        def same(k, scale):
            got = bench.cache.k.view(I8)[p, :, 0].cpu()
            assert torch.equal(got.transpose(0, 1), k)
            assert torch.equal(bench.cache.v.view(I8)[p, :, 0].cpu().permute(2, 0, 1), k)
            assert torch.equal(bench.cache.k_scale[p, :, 0].cpu(), scale)
            assert torch.equal(bench.cache.v_scale[p, :, 0].cpu(), scale)

        first = torch.cat([code(a * (1 / s)[None, :, None]), torch.zeros(11, 2, 32, dtype=I8)])
        same(first, s)
        bench.append([4], rows=(b, b))
        s2 = torch.maximum(s, b.abs().amax((0, 2)) * torch.tensor(1.0 / top, dtype=F32))
        old = first[:5].view(fmt).float() * (s * (1 / s2))[None, :, None]
        second = torch.cat([code(old), code(b * (1 / s2)[None, :, None]), torch.zeros(7, 2, 32, dtype=I8)])
        same(second, s2)


@pytest.mark.parametrize("fmt", [I8, F8], ids=["int8", "fp8"])
def test_append_zero_tiny_and_not_finite(fmt):
    """All-zero blocks hold zeros; values under the smallest normal scale vanish; NaN and infinity poison their block
    of 16 tokens and head, and nothing else."""
    bench = Bench(1, 2, 64, 32, 64, fmt)
    z = torch.zeros(16, 2, 64)
    bench.append([16], rows=(z, z + 1e-41))
    assert (bench.held()[0] == 0).all() and (bench.held()[1] == 0).all()
    k, v = normal(bench.g, 20, 2, 64), normal(bench.g, 20, 2, 64)
    k[3, 1, 5], v[18, 0, 0] = float("nan"), float("inf")
    kv = torch.tensor([36], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    bench.cache.append(k.to(DEV), v.to(DEV), kv, bench.pages, cu_q=cu, max_q=20)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    gk, gv = bench.cache.read(zero, kv, bench.pages, 36, dtype=F32)
    for g, blk, head in ((gk, slice(16, 32), 1), (gv, slice(32, 36), 0)):
        assert torch.isnan(g[0, blk, head]).all()
        g[0, blk, head] = 0
        assert torch.isfinite(g).all()
    q = normal(bench.g, 1, 4, 64, dtype=BF).to(DEV)
    out = bench.cache.attend(q, kv, bench.pages)
    assert torch.isnan(out[0]).all()                       # heads 2, 3 read the poisoned K block, 0, 1 the V block
    for n, bad in ((16, []), (32, [2, 3])):                # before the poisoned blocks; K's only
        out = bench.cache.attend(q, torch.tensor([n], dtype=torch.int32, device=DEV), bench.pages)
        assert [j for j in range(4) if torch.isnan(out[0, j]).any()] == bad
    # the poison leaves when the block is begun anew
    bench.len = [16]
    bench.append([20], rows=(normal(bench.g, 20, 2, 64), normal(bench.g, 20, 2, 64)))
    bench.check()


def test_append_idle_cut_back_and_missing_pages():
    bench = Bench(3, 2, 32, 16, 64, I8)
    bench.append([20, 33, 5])
    bench.append([1, 1, 1])
    # cut back by a few tokens inside and across blocks, then continued: the scale stays at least the old one
    bench.len = [18, 16, 0]
    bench.append([3, 2, 1])
    bench.check(times=3)
    # an idle slot brings a row that is not stored; a page table entry outside the pool drops its tokens
    kept = bench.cache.k.view(I8).clone()
    kv = torch.tensor([0, 19, 0], dtype=torch.int32, device=DEV)
    pages = bench.pages.clone()
    pages[1, 1] = bench.n_pages
    x = normal(bench.g, 3, 2, 32).to(DEV)
    q = bench.cache.append(x, x, kv, pages, q=x, inv_freq=attention.rope_frequencies(32)[0])
    assert torch.equal(bench.cache.k.view(I8), kept)
    want = ref.turn(x.cpu(), torch.tensor([-1, 18, -1]), attention.rope_frequencies(32, device="cpu")[0])
    within(q, want, turn_bound(x.cpu(), want, 1.0, F32), "q")


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_append_fused_projection(io, shift):
    """q, k and v as parts of one projection, aligned or not; q in place."""
    g = gen(31 + shift)
    H, G, D, T = 4, 2, 64, 21
    buf = normal(g, T, (H + 2 * G) * D + 16, dtype=io).to(DEV)
    x = buf[:, shift:shift + (H + 2 * G) * D].view(T, H + 2 * G, D)
    q, k, v = x[:, :H], x[:, H:H + G], x[:, H + G:]
    f = attention.rope_frequencies(D)[0]
    bench = Bench(1, G, D, 16, 32, I8)
    plain = bench.cache
    other = attention.KVCache.empty(bench.n_pages, 16, G, D)
    kv, cu = torch.tensor([T], dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV)
    q1 = plain.append(k.contiguous(), v.contiguous(), kv, bench.pages, cu_q=cu, max_q=T, q=q.contiguous(), inv_freq=f)
    q2 = other.append(k, v, kv, bench.pages, cu_q=cu, max_q=T, q=q, q_out=q, inv_freq=f)
    assert torch.equal(q1, q2) and q2.data_ptr() == q.data_ptr()
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    for a, b in zip(plain.read(zero, kv, bench.pages, T), other.read(zero, kv, bench.pages, T)):
        assert torch.equal(a, b)


def test_read_ranges():
    """Ranges that begin inside a block, pass the end, or lie before the first position; counts above the room."""
    bench = Bench(4, 2, 48, 32, 96, F8)
    bench.append([70, 40, 96, 3])
    whole = [bench.held(BF), bench.held(F32)]
    first = torch.tensor([5, 0, 90, -4], dtype=torch.int32, device=DEV)
    count = torch.tensor([37, 40, 300, 7], dtype=torch.int32, device=DEV)
    for dt, (hk, hv) in zip((BF, F32), whole):
        k, v = bench.cache.read(first, count, bench.pages, 45, dtype=dt)
        for got, held in ((k, hk), (v, hv)):
            assert torch.equal(got[0, :37], held[0, 5:42]) and (got[0, 37:] == 0).all()
            assert torch.equal(got[1, :40], held[1, :40]) and (got[1, 40:] == 0).all()
            assert torch.equal(got[2, :6], held[2, 90:96]) and (got[2, 6:] == 0).all()
            assert (got[3, :4] == 0).all() and torch.equal(got[3, 4:7], held[3, :3])
    k, v = bench.cache.read(first, count, bench.pages, 0)
    assert k.shape == (4, 0, 2, 48) and v.shape == k.shape


# ---------------------------------------------------------------------------------------------------------- attention

ATTEND = [  # kv heads, q heads, dim, page, fmt, io, lens, rows per sequence, causal, window
    (1, 1, 64, 16, I8, BF, [1, 2, 15, 16, 17], [1] * 5, True, 0),
    (2, 8, 128, 64, I8, BF, [63, 64, 65, 300, 0], [1] * 5, True, 0),
    (4, 4, 128, 32, F8, F32, [127, 128, 129, 1], [1] * 4, True, 0),
    (1, 40, 64, 16, F8, BF, [33, 200], [1] * 2, True, 0),                # 40 heads on one key head
    (2, 6, 80, 16, I8, F32, [100, 37, 5], [3, 0, 5], True, 0),
    (2, 4, 256, 64, F8, BF, [90, 130], [7, 2], True, 0),
    (3, 3, 32, 128, I8, F32, [70, 257], [70, 19], True, 0),              # a whole prompt; the end of one
    (2, 4, 96, 16, I8, BF, [150, 64], [33, 64], False, 0),
    (1, 2, 16, 16, I8, F32, [90, 3], [2, 3], True, 1),                   # a window of the row itself
    (2, 2, 64, 32, F8, BF, [300, 40, 0, 129], [1, 1, 1, 1], True, 64),
    (1, 8, 128, 16, I8, BF, [400, 500], [65, 20], True, 100),
    (1, 3, 48, 64, F8, F32, [3, 9], [5, 9], True, 0),                    # more rows than tokens held: positions < 0
    (2, 32, 192, 32, I8, F32, [77], [9], True, 30),
    (1, 16, 112, 16, F8, BF, [1500], [1], True, 0),
    (2, 4, 128, 64, F8, BF, [520, 130], [200, 130], True, 0),
    (2, 8, 64, 64, I8, BF, [700, 310, 64], [130, 310, 64], True, 0),
    (1, 1, 128, 128, I8, BF, [1100], [1100], True, 0),
    (2, 4, 64, 16, F8, BF, [600, 80], [150, 80], True, 90),
    (1, 6, 128, 32, I8, BF, [333, 290], [100, 290], False, 0),
]


def a_bench(case, room=None):
    kv, H, D, page, fmt, io, lens, n, causal, window = case
    bench = Bench(len(lens), kv, D, page, max(lens + [1]) if room is None else room, fmt, seed=D + H)
    bench.append(list(lens))
    return bench, normal(bench.g, sum(n), H, D, dtype=io)


@pytest.mark.parametrize("bound", ["tight", "loose"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(str(v) for v in c))
def test_attend(case, bound):
    """Against 64 bits, with the launch sized tightly and by a loose bound (other tiles and splits)."""
    kv, H, D, page, fmt, io, lens, n, causal, window = case
    bench, q = a_bench(case, room=None if bound == "tight" else max(lens) + 3000)
    tight = dict(max_kv=max(lens)) if bound == "tight" else dict(max_q=max(n) + 500 if n != [1] * len(n) else 1)
    bench.attend(q, n, io, causal, window, **tight)


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("batch,rows", [(300, 1), (40, 9), (2100, 1)])
def test_attend_many_ragged_sequences(batch, rows, window):
    """Lengths from nothing to many tiles dealt out among the workgroups: more sequences than threads, several row
    tiles a sequence, idle slots between; and more sequences than a workgroup keeps account of."""
    g = gen(batch)
    top = 1300 if batch < 1000 else 1100
    lens = torch.randint(0, 90 if batch > 1000 else top, (batch,), generator=g).tolist()
    lens[3], lens[batch // 2], lens[-1], lens[1] = top, 0, 0, top
    bench = Bench(batch, 1, 16, 16, top, I8, seed=batch)
    bench.append(lens)
    q = normal(g, batch * rows, 4, 16, dtype=F32)
    bench.attend(q, [rows] * batch, F32, window=window)


def test_attend_scale_and_peaks():
    """Large scores: one key takes all; a zero scale gives the mean."""
    for io in (BF, F32):
        case = (1, 2, 64, 16, I8, io, [200], [4], True, 0)
        bench, q = a_bench(case)
        bench.attend(q, [4], io, scale=30.0)
        bench.attend(q, [4], io, scale=0.0)
        bench.attend(q, [4], io, scale=-0.3)


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 70])
def test_attend_scores_that_jump(rows, dim, io):
    """One key a sequence, each place of a tile in turn, lies 2^58 above all before it; then the scores fall again.
    (Blocks share a scale, so the loud key's neighbours lose their small values: the reference reads what is held.)"""
    L, at = 200, torch.arange(64) + 64
    bench = Bench(64, 1, dim, 16, 208, F8, seed=dim)
    u = torch.zeros(dim)
    u[::8] = 1.0
    k = 0.05 * normal(bench.g, 64, L, 1, dim)
    k[torch.arange(64), at, 0] += 40.0 / (dim / 8) * u
    k[:, 170:] -= 3.0 / (dim / 8) * u
    v = normal(bench.g, 64, L, 1, dim)
    bench.append([L] * 64, rows=(k.reshape(-1, 1, dim), v.reshape(-1, 1, dim)))
    q = (u + 0.05 * normal(bench.g, 64 * rows, 2, dim)).to(io)
    bench.attend(q, [rows] * 64, io, scale=1.0)


@pytest.mark.parametrize("dim", [64, 128])
def test_attend_scores_that_jump_in_prompts(dim):
    """The same where the rows are most of the keys (half the rows a workgroup)."""
    test_attend_scores_that_jump(150, dim, BF)


def test_attend_missing_pages():
    """Keys of pages outside the pool are absent, at the start, inside, and all of a sequence's."""
    for n in ([1, 1, 1], [40, 130, 20]):
        case = (2, 4, 64, 16, F8, BF, [150, 140, 20], n, True, 0)
        bench, q = a_bench(case)
        bench.attend(q, n, BF, gone=[(0, 0), (0, 3), (1, 5), (2, 0), (2, 1)])


def test_attend_strided_queries():
    g = gen(4)
    for io in (BF, F32):
        for n, shift in (([1, 1], 0), ([1, 1], 1), ([150, 3], 0), ([150, 3], 1)):
            case = (2, 4, 64, 16, I8, io, [150, 77], n, True, 0)
            bench, _ = a_bench(case)
            buf = normal(g, sum(n), 7 * 64 + 8, dtype=io).to(DEV)
            q = buf[:, shift:shift + 6 * 64].view(sum(n), 6, 64)[:, 1:5]
            bench.attend(q, n, io)
            bench.attend(q.transpose(0, 1).contiguous().transpose(0, 1), n, io)


def test_attend_rows_beyond_the_bounds_stay_in_bounds():
    """Lengths and pages that make no sense are held inside the buffers (and their rows see what is left)."""
    case = (1, 2, 64, 16, I8, BF, [100, 60], [1, 1], True, 0)
    bench, q = a_bench(case)
    kv = torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32, device=DEV)
    out, lse = bench.cache.attend(q.to(DEV), kv, bench.pages, lse=True)
    assert (out[1] == 0).all() and torch.isinf(lse[1]).all()
    cu = torch.tensor([0, 9, 4], dtype=torch.int32, device=DEV)
    bench.cache.attend(q.to(DEV), bench.kv_len(), bench.pages, cu_q=cu, max_q=2)
    bench.cache.append(q[:, :1].to(DEV).contiguous(), q[:, :1].to(DEV).contiguous(), kv, bench.pages, cu_q=cu, max_q=2)
    torch.cuda.synchronize()


def test_attend_empty_calls():
    bench = Bench(2, 1, 64, 16, 32, I8)
    none = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert bench.cache.attend(none, bench.kv_len(), bench.pages, cu_q=cu, max_q=0).shape == (0, 2, 64)
    assert bench.cache.append(none[:, :1], none[:, :1], bench.kv_len(), bench.pages, cu_q=cu, max_q=0) is None
    q = normal(bench.g, 2, 2, 64, dtype=BF).to(DEV)                      # nothing held by anybody
    for n_pages in (0, 2):
        out, lse = bench.cache.attend(q, bench.kv_len(), bench.pages[:, :n_pages].contiguous(), lse=True)
        assert (out == 0).all() and (lse == -math.inf).all()
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    assert bench.cache.attend(none, e, torch.empty(0, 3, dtype=torch.int32, device=DEV)).shape == (0, 2, 64)


def test_attend_same_bits_again_and_alone():
    """A call's bits do not depend on the call before, on the other sequences, or on the stream."""
    case = (2, 8, 128, 64, I8, BF, [700, 300, 1500], [1, 1, 1], True, 0)
    bench, q = a_bench(case)
    qd = q.to(DEV)
    a = bench.cache.attend(qd, bench.kv_len(), bench.pages)
    side = torch.cuda.Stream()
    kv = bench.kv_len()
    side.wait_stream(torch.cuda.current_stream())
    b = bench.cache.attend(qd, kv, bench.pages, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)
    assert torch.equal(a, bench.cache.attend(qd, kv, bench.pages))


def test_cache_beyond_32_bit_offsets():
    """Pages whose codes lie past 4 GiB of each pool."""
    D, heads, page = 128, 2, 64
    n = (1 << 32) // (D * heads * page) + 40
    cache = attention.KVCache.empty(n, page, heads, D, dtype=I8)
    g = gen(8)
    k, v = normal(g, 100, heads, D, dtype=BF), normal(g, 100, heads, D, dtype=BF)
    q = normal(g, 100, 4, D, dtype=BF).to(DEV)
    cu, kv = torch.tensor([0, 100], dtype=torch.int32, device=DEV), torch.tensor([100], dtype=torch.int32, device=DEV)
    low, high = (torch.tensor([p], dtype=torch.int32, device=DEV) for p in ([3, 1], [n - 1, n - 3]))
    got = []
    for pages in (low, high):
        cache.append(k.to(DEV), v.to(DEV), kv, pages, cu_q=cu, max_q=100)
        got.append((cache.attend(q, kv, pages, cu_q=cu, max_q=100), cache.attend(q[:1], kv, pages),
                    *cache.read(torch.zeros_like(kv), kv, pages, 100)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(cache.k[3], cache.k[n - 1]) and torch.equal(cache.v[1], cache.v[n - 3])


def test_decode_in_a_graph():
    """append + attend captured once, replayed as the lengths grow on the device, against the eager calls."""
    H, G, D, page, steps = 8, 2, 64, 16, 6
    f = attention.rope_frequencies(D)[0]

    def fresh():
        bench = Bench(2, G, D, page, 128, I8, seed=1)
        bench.append([30, 77])
        return bench

    g = gen(77)
    xs = [normal(g, 2, H + 2 * G, D, dtype=BF).to(DEV) for _ in range(steps)]
    eager, cap = fresh(), fresh()
    kv_e, kv_c = eager.kv_len(), cap.kv_len()
    x = torch.empty_like(xs[0])

    def step(bench, kv, x):
        kv.add_(1)
        q = bench.cache.append(x[:, H:H + G], x[:, H + G:], kv, bench.pages, q=x[:, :H], inv_freq=f)
        return bench.cache.attend(q, kv, bench.pages)

    x.copy_(xs[0])
    keep = [t.clone() for t in (cap.cache.k.view(I8), cap.cache.v.view(I8), cap.cache.k_scale, cap.cache.v_scale, kv_c)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap, kv_c, x)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out = step(cap, kv_c, x)
    for t, o in zip((cap.cache.k.view(I8), cap.cache.v.view(I8), cap.cache.k_scale, cap.cache.v_scale, kv_c), keep):
        t.copy_(o)
    for j in range(steps):
        x.copy_(xs[j])
        graph.replay()
        want = step(eager, kv_e, xs[j])
        torch.cuda.synchronize()
        assert torch.equal(out, want), j
        torch.randn(1000, device=DEV).sum()                               # the program's own work in between


def test_prompt_then_steps_agree_with_one_prompt():
    """A prompt attended in one piece, in two, and its tail token by token see the same cache."""
    H, G, D, L = 4, 2, 64, 150
    g = gen(21)
    x = normal(g, L, H + 2 * G, D, dtype=F32).to(DEV)
    f = attention.rope_frequencies(D)[0]
    bench = Bench(1, G, D, 32, 160, I8)
    outs = []

    def feed(lo, hi):
        kv = torch.tensor([hi], dtype=torch.int32, device=DEV)
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV)
        y = x[lo:hi]
        q = bench.cache.append(y[:, H:H + G], y[:, H + G:], kv, bench.pages, cu_q=cu, max_q=hi - lo, q=y[:, :H], inv_freq=f)
        return q, bench.cache.attend(q, kv, bench.pages, cu_q=cu, max_q=hi - lo)

    q, whole = feed(0, L)
    kv, cu = torch.tensor([L], dtype=torch.int32, device=DEV), torch.tensor([0, L], dtype=torch.int32, device=DEV)
    # the same cache, its rows asked for in pieces: fp32 sums in another order
    for lo, hi in ((0, 96), (96, 149), (149, 150)):
        part = torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV)
        outs.append(bench.cache.attend(q[lo:hi], torch.tensor([hi], dtype=torch.int32, device=DEV), bench.pages,
                                       cu_q=part, max_q=hi - lo))
    k, v = bench.held() if bench.len != [0] else bench.cache.read(torch.zeros_like(kv), kv, bench.pages, L, dtype=F32)
    o, _, mag, top = ref.attend(q.cpu(), torch.arange(L), k[0].cpu(), v[0].cpu(), 1 / math.sqrt(D))
    bound = ref.attend_bound(o, mag, top, D, L, F32)
    within(whole, o, bound, "whole")
    within(torch.cat(outs), o, bound, "pieces")
