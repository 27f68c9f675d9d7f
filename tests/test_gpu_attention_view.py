"""Attention over the paged cache under a window with sinks, and with first pages that sequences hold together, against
64 bits over the values that the cache holds."""
import math

import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests import attn_ref as ref
from tests.test_gpu_attention import BF, DEV, F32, F8, I8, Bench, gen, normal, within

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def reference(q, k, v, scale, ok):
    """Rows q [n][heads][dim] over k, v [len][kv heads][dim], row t seeing the keys ok[t]: out, lse, sum p |v|, the largest
    scale sum |q| |k|."""
    n, H, D = q.shape
    G = H // k.shape[1]
    qd, kd, vd = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    s = torch.matmul(qd.transpose(0, 1), kd.permute(1, 2, 0).contiguous()) * scale
    big = torch.matmul(qd.abs().transpose(0, 1), kd.abs().permute(1, 2, 0).contiguous()) * abs(scale)
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:2], -math.inf, dtype=torch.float64)
    p = torch.where(ok & ok.any(-1, keepdim=True), (s - lse[..., None]).exp(), torch.zeros_like(s))
    vt = vd.transpose(0, 1)
    top = big.masked_fill(~ok, 0.0).amax(-1) if s.shape[-1] else torch.zeros(H, n, dtype=torch.float64)
    return (torch.matmul(p, vt).transpose(0, 1), lse.transpose(0, 1), torch.matmul(p, vt.abs()).transpose(0, 1),
            top.transpose(0, 1))


def visible(pos, length, causal, window, sinks):
    at = torch.arange(length)[None, :]
    ok = torch.ones(len(pos), length, dtype=torch.bool)
    if causal:
        ok &= at <= pos[:, None]
    if window:
        ok &= (at > pos[:, None] - window) | (at < sinks)
    return ok


class View(Bench):
    """Sequences in pages of their own; those of a group take their first pages from the group's longest sequence (a shorter
    one's may never have been written)."""

    def look(self, q, n, io, causal=True, window=0, sinks=0, starts=None, counts=None, lens=None, bound=None, drop=False,
             lse=True, cu=None, scale=None, gone=()):
        lens = self.len if lens is None else lens
        pages = self.pages.clone()
        prefix, first, of = None, [(None, 0)] * self.batch, [None] * self.batch
        if starts is not None:
            wide = max(counts + [1])
            shared = torch.full((len(counts), wide), -7, dtype=torch.int32, device=DEV)
            for g, c in enumerate(counts):
                members = range(starts[g], starts[g + 1])
                if not members:
                    continue
                donor = max(members, key=lambda i: self.len[i])
                shared[g, :c] = self.pages[donor, :c]
                for i in members:
                    first[i] = (donor, c * self.page)
                    of[i] = g
                    pages[i, :c] = self.spare[0].item() if i % 2 else -3    # a page of NaN codes and scales, or none
            for g, p in gone:
                shared[g, p] = -1
            prefix = attention.SharedPrefix(shared, ints(counts), ints(starts) if len(starts) != 2 or starts != [0, self.batch]
                                            else None)
        if drop:    # pages that hold neither first tokens nor any row's window: given back, in other hands
            for i, c in enumerate(n):
                low = max(0, lens[i] - c - window + 1)
                for j in range(pages.shape[1]):
                    if j * self.page >= sinks and (j + 1) * self.page <= low:
                        pages[i, j] = self.spare[0].item() if j % 2 else -1
        if cu is None and n != [1] * self.batch:
            cu = ints([sum(n[:j]) for j in range(len(n) + 1)])
        kw = dict(max_q=max(n + [1]), max_kv=max(lens + [1])) if bound is None else bound
        got = self.cache.attend(q.to(DEV) if not q.is_cuda else q, ints(lens), pages, cu_q=cu, causal=causal, window=window,
                                sinks=sinks, prefix=prefix, lse=lse, scale=scale, **kw)
        out, l = got if lse else (got, None)
        kd, vd = (x.cpu() for x in self.held())
        at = 0
        for i, c in enumerate(n):
            L, (g0, p) = lens[i], first[i]
            p = min(p, L)
            k = kd[i, :L] if not p else torch.cat([self.first(kd, g0, p), kd[i, p:L]])
            v = vd[i, :L] if not p else torch.cat([self.first(vd, g0, p), vd[i, p:L]])
            ok = visible(torch.arange(L - c, L), L, causal, window, sinks)
            for g, pg in gone:
                if of[i] == g:
                    ok[:, pg * self.page:min(p, (pg + 1) * self.page)] = False
            o, z, mag, top = reference(q[at:at + c].cpu(), k, v, 1 / math.sqrt(self.dim) if scale is None else scale, ok)
            within(out[at:at + c], o, ref.attend_bound(o, mag, top, self.dim, L, io), f"out {i}")
            if lse:
                zb = 2.0 ** -24 * (L + (self.dim + 4) * top + 8) * 2 + z.abs() * 2.0 ** -22 + 1e-6
                y = l[at:at + c].cpu().double()
                assert torch.equal(torch.isinf(y), torch.isinf(z)) and (((y - z).abs() <= zb) | torch.isinf(z)).all(), i
            at += c
        return out

    def first(self, held, g0, p):
        return held[g0, :p]


def bench_of(kv, D, page, fmt, lens, room=None, seed=0):
    b = View(len(lens), kv, D, page, max(lens + [1]) if room is None else room, fmt, seed=seed + D, spare=2)
    b.append(list(lens))
    return b


# ---------------------------------------------------------------------------------------------------------- sinks

SINKS = [  # kv heads, q heads, dim, page, fmt, io, lens, rows per sequence, window, sinks
    (1, 1, 64, 16, I8, BF, [1, 2, 15, 40, 300], [1] * 5, 1, 1),
    (2, 8, 128, 64, I8, BF, [63, 400, 1500, 0, 700], [1] * 5, 100, 4),
    (4, 4, 128, 32, F8, F32, [127, 1128, 129, 1], [1] * 4, 64, 64),
    (2, 6, 80, 16, I8, F32, [900, 37, 5], [3, 0, 5], 130, 65),
    (2, 4, 256, 64, F8, BF, [90, 730], [7, 2], 50, 17),
    (3, 3, 32, 128, I8, F32, [70, 957], [70, 19], 33, 200),          # more sinks than some rows' whole past
    (1, 40, 64, 16, F8, BF, [333, 2000], [1] * 2, 257, 5),
    (1, 8, 128, 16, I8, BF, [1400, 500], [65, 20], 100, 3),
    (2, 4, 96, 16, I8, BF, [1150, 64], [33, 64], 40, 16),
    (2, 32, 192, 32, I8, F32, [1077], [9], 30, 1),
    (2, 4, 128, 64, F8, BF, [1520, 130], [200, 130], 64, 70),
    (2, 8, 64, 64, I8, BF, [1700, 310, 64], [130, 310, 64], 128, 10),
    (1, 1, 128, 128, I8, BF, [1100], [1100], 90, 1),
    (2, 4, 64, 16, F8, F32, [1600, 80], [150, 80], 256, 128),
    (1, 2, 256, 16, I8, F32, [700], [90], 40, 33),
    (1, 3, 48, 64, F8, F32, [3, 9], [5, 9], 2, 1),                   # more rows than tokens held: positions < 0
]


@pytest.mark.parametrize("bound", ["tight", "loose"])
@pytest.mark.parametrize("case", SINKS, ids=lambda c: "-".join(str(v) for v in c))
def test_sinks(case, bound):
    """Pages in between are given back; the launch sized tightly and by a loose bound."""
    kv, H, D, page, fmt, io, lens, n, window, sinks = case
    b = bench_of(kv, D, page, fmt, lens, room=None if bound == "tight" else max(lens) + 3000, seed=H)
    q = normal(b.g, sum(n), H, D, dtype=io)
    b.look(q, n, io, window=window, sinks=sinks, drop=True,
           bound=None if bound == "tight" else dict(max_q=max(n) + 500 if n != [1] * len(n) else 1))


@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("sinks", [1, 15, 16, 17, 63, 64, 65, 128, 130, 300, 449, 450, 451, 2 ** 40])
def test_sinks_at_every_edge(sinks, rows):
    """Sinks that end inside and at the ends of blocks and tiles, that meet the window, and that hold everything."""
    b = bench_of(2, 64, 16, I8, [600, 512, 70], seed=sinks % 100)
    q = normal(b.g, 3 * rows, 4, 64, dtype=F32)
    b.look(q, [rows] * 3, F32, window=150, sinks=sinks)


def test_sinks_meet_the_plain_calls():
    """No sinks, sinks without a window, and sinks of everything are the calls without them."""
    for n, io in (([1, 1], BF), ([120, 60], BF), ([3, 9], F32)):
        b = bench_of(2, 128, 64, F8, [900, 400])
        q = normal(b.g, sum(n), 8, 128, dtype=io).to(DEV)
        cu = ints([0, n[0], sum(n)])
        kw = dict(cu_q=cu, max_q=max(n), lse=True)
        plain = lambda **k: b.cache.attend(q, b.kv_len(), b.pages, **kw, **k)  # noqa: E731
        for x, y in ((plain(), plain(sinks=70)), (plain(window=100), plain(window=100, sinks=0)),
                     (plain(), plain(window=2000, sinks=3))):
            assert all(torch.equal(s, t) for s, t in zip(x, y)) or not torch.equal(x[0], x[0])
        whole, every = plain(), plain(window=50, sinks=900)
        for s, t in zip(whole, every):
            assert (s.float() - t.float()).abs().max() <= 2.0 ** -7 * s.float().abs().max()


@pytest.mark.parametrize("batch,rows", [(300, 1), (40, 9), (2100, 1)])
def test_sinks_of_many_ragged_sequences(batch, rows):
    g = gen(batch)
    top = 1300 if batch < 1000 else 1100
    lens = torch.randint(0, 90 if batch > 1000 else top, (batch,), generator=g).tolist()
    lens[3], lens[batch // 2], lens[-1], lens[1] = top, 0, 0, top
    b = bench_of(1, 16, 16, I8, lens, seed=batch)
    q = normal(g, batch * rows, 4, 16, dtype=F32)
    b.look(q, [rows] * batch, F32, window=200, sinks=20, drop=True)


# ---------------------------------------------------------------------------------------------------------- prefixes

PREFIX = [  # kv heads, q heads, dim, page, fmt, io, lens, rows per sequence, group starts, pages of each prefix
    (2, 8, 128, 64, I8, BF, [700, 650, 641, 900], [1] * 4, [0, 4], [10]),
    (1, 1, 64, 16, F8, F32, [40, 33, 35], [1] * 3, [0, 3], [2]),
    (2, 6, 80, 16, I8, F32, [100, 137, 55, 290, 0, 310, 20], [3, 0, 5, 1, 1, 2, 2], [0, 3, 6, 7], [3, 17, 1]),
    (4, 16, 128, 32, F8, BF, [1100] * 9 + [1060], [1] * 10, [0, 10], [33]),
    (2, 4, 256, 64, F8, BF, [290, 330, 270], [7, 2, 1], [0, 3], [4]),
    (1, 8, 64, 16, I8, BF, [500, 480, 470, 600, 30, 700, 690], [1] * 7, [1, 4, 4, 7], [29, 5, 31]),  # some share nothing
    (2, 4, 96, 16, I8, BF, [350, 264, 300], [33, 64, 20], [0, 3], [16]),
    (2, 4, 64, 16, F8, BF, [600, 680, 590], [150, 80, 1], [0, 2, 3], [32, 30]),
    (1, 4, 128, 64, F8, F32, [800, 700], [100, 60], [0, 2], [10]),
    (2, 2, 192, 32, I8, F32, [200, 230, 220], [9, 1, 4], [0, 3], [6]),
    (1, 2, 16, 128, I8, F32, [300, 257], [2, 1], [0, 2], [2]),
    (2, 4, 64, 16, I8, BF, [64, 64, 48, 40, 7, 0], [1] * 6, [0, 6], [4]),      # nothing of their own; shorter than the prefix
    (1, 3, 32, 16, F8, F32, [64, 60, 70, 9], [4, 6, 9, 9], [0, 4], [4]),       # rows inside the prefix
    (2, 8, 64, 64, I8, BF, [500, 400], [1, 1], [0, 2], [0]),                   # an empty prefix
]


@pytest.mark.parametrize("bound", ["tight", "loose"])
@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(str(v) for v in c))
def test_prefix(case, bound):
    kv, H, D, page, fmt, io, lens, n, starts, counts = case
    b = bench_of(kv, D, page, fmt, lens, room=None if bound == "tight" else max(lens) + 2500, seed=H)
    q = normal(b.g, sum(n), H, D, dtype=io)
    b.look(q, n, io, starts=starts, counts=counts,
           bound=None if bound == "tight" else dict(max_q=max(n) + 300 if n != [1] * len(n) else 1))
    if n != [1] * len(n) and bound == "loose":
        b.look(q, n, io, starts=starts, counts=counts, bound={}, lse=False)


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,H,kv,D,tail", [(16, 8, 2, 128, 300), (70, 8, 2, 64, 90), (150, 4, 1, 128, 40), (33, 16, 4, 80, 700),
                                               (20, 2, 2, 256, 200), (600, 8, 8, 32, 20)])
def test_prefix_of_many(batch, H, kv, D, tail, io):
    """Batches behind one long prompt: few rows to many, own lengths from nothing to some hundreds, idle slots."""
    g = gen(batch + D)
    page, count = 64, 24
    lens = (count * page + torch.randint(1, tail, (batch,), generator=g)).tolist()
    lens[1], lens[-1], lens[2] = 0, 0, count * page
    b = bench_of(kv, D, page, I8 if batch % 2 else F8, lens, seed=batch)
    q = normal(g, batch, H, D, dtype=io)
    b.look(q, [1] * batch, io, starts=[0, batch], counts=[count])


@pytest.mark.parametrize("batch,per", [(96, 3), (64, 16), (300, 100)])
def test_prefix_in_groups(batch, per):
    """Groups with prefixes of their own, of 0 pages to many, drafts of some rows among them."""
    g = gen(batch)
    page = 16
    starts = list(range(0, batch + 1, per))
    counts = torch.randint(0, 60, (len(starts) - 1,), generator=g).tolist()
    n = torch.randint(0, 4, (batch,), generator=g).tolist()
    lens = [counts[min(i // per, len(counts) - 1)] * page + a for i, a in enumerate(torch.randint(4, 120, (batch,), generator=g).tolist())]
    b = bench_of(2, 64, page, I8, lens, seed=per)
    q = normal(g, sum(n), 8, 64, dtype=BF)
    b.look(q, n, BF, starts=starts, counts=counts)
    b.look(q, n, BF, starts=starts, counts=counts, causal=False, bound={})


def test_prefix_with_a_window_and_sinks():
    for n, window, sinks in (([1] * 5, 300, 0), ([1] * 5, 100, 20), ([40] * 5, 130, 70), ([2] * 5, 1000, 5)):
        b = bench_of(2, 64, 16, F8, [500, 420, 700, 600, 418])
        q = normal(b.g, sum(n), 4, 64, dtype=BF)
        b.look(q, n, BF, window=window, sinks=sinks, starts=[0, 3, 5], counts=[26, 20])


def test_prefix_pages_that_are_absent():
    """Shared pages outside the pool hold no keys, for every sequence of their group and no other."""
    for n in ([1] * 6, [30] * 6):
        b = bench_of(2, 64, 16, I8, [300, 280, 290, 270, 310, 330])
        q = normal(b.g, sum(n), 4, 64, dtype=F32)
        b.look(q, n, F32, starts=[0, 3, 6], counts=[15, 12], gone=[(0, 0), (0, 7), (1, 11)])


def test_prefix_loud_keys():
    """Scores that take all in the prefix for some rows, in their own keys for others; scales of V far apart."""
    D, page, count = 64, 16, 8
    lens = [count * page + 30 + i for i in range(6)]
    for io in (BF, F32):
        b = View(6, 1, D, page, max(lens), I8, seed=3)
        k = 0.05 * normal(b.g, sum(lens), 1, D)
        v = normal(b.g, sum(lens), 1, D)
        at = 0
        for i, l in enumerate(lens):
            k[at + (20 if i == 0 else count * page + 3)] += 8.0 if i % 2 else 0.0
            k[at + 20] += 8.0 if i == 0 else 0.0
            v[at:at + count * page] *= 2.0 ** -20 if i == 0 else 1.0
            at += l
        b.append(list(lens), rows=(k, v))
        q = normal(b.g, 6, 2, D, dtype=io) + 1
        b.look(q, [1] * 6, io, starts=[0, 6], counts=[count], scale=1.0)


def test_prefix_devices_arrays_out_of_range_stay_in_bounds():
    """Counts, starts and pages that make no sense are held inside the arrays."""
    b = bench_of(1, 64, 16, I8, [100, 60, 80, 70])
    q = normal(b.g, 4, 2, 64, dtype=BF).to(DEV)
    kv = b.kv_len()
    for starts, count, table in (([0, 9, -4], [2 ** 31 - 1, -5], [[3, 2 ** 31 - 1], [-9, 10 ** 6]]),
                                 ([-2 ** 31, 2, 2 ** 31 - 1], [1, 2], [[0, 1], [2, 3]]), ([4, 4, 4], [2, 2], [[0, 1], [2, 3]]),
                                 ([3, 1, 2], [2, 2], [[0, 1], [2, 3]])):
        p = attention.SharedPrefix(ints(table), ints(count), ints(starts))
        b.cache.attend(q, kv, b.pages, prefix=p)
        b.cache.attend(q, ints([0, 0, 0, 0]), b.pages, prefix=p)
        b.cache.attend(q, ints([2 ** 31 - 1, -3, 5, 9]), b.pages, prefix=p, cu_q=ints([0, 3, 1, 9, 4]), max_q=3)
        b.cache.attend(q.repeat(60, 1, 1), kv, b.pages, prefix=p, cu_q=ints([0, 100, 150, 220, 240]), max_q=100)
    torch.cuda.synchronize()
    p = attention.SharedPrefix(ints([[3, 1]]), ints([-5]))
    assert torch.equal(b.cache.attend(q, kv, b.pages, prefix=p), b.cache.attend(q, kv, b.pages, prefix=attention.SharedPrefix(
        ints([[3, 1]]), ints([0]))))


def test_prefix_beyond_max_kv_and_max_q():
    """Bounds below what is there: keys past max_kv are not seen, rows past max_q keep what they held."""
    b = bench_of(2, 64, 16, F8, [300, 280, 260])
    n = [5, 2, 7]
    q = normal(b.g, sum(n), 4, 64, dtype=F32)
    shared = b.pages[:1, :15].contiguous()
    p = attention.SharedPrefix(shared, ints([15]))
    cu = ints([0, 5, 7, 14])
    out = torch.full((14, 4, 64), 7.0, device=DEV)
    b.cache.attend(q.to(DEV), b.kv_len(), b.pages, cu_q=cu, max_q=3, prefix=p, out=out)
    whole = b.cache.attend(q.to(DEV), b.kv_len(), b.pages, cu_q=cu, max_q=7, prefix=p)
    rows = [0, 1, 2, 5, 6, 7, 8, 9]
    left = [3, 4, 10, 11, 12, 13]
    assert (out[left] == 7.0).all()
    assert (out[rows] - whole[rows]).abs().max() <= 2.0 ** -18 * whole.abs().max()
    short = b.cache.attend(q.to(DEV), b.kv_len(), b.pages, cu_q=cu, max_q=7, max_kv=100, prefix=p)
    kd, vd = (x.cpu() for x in b.held())
    o, _, mag, top = reference(q, kd[0, :100], vd[0, :100], 1 / 8, torch.ones(14, 100, dtype=torch.bool))
    within(short, o, ref.attend_bound(o, mag, top, 64, 100, F32), "short")


# ---------------------------------------------------------------------------------------------------------- calls

@pytest.mark.parametrize("kind", ["sinks", "prefix"])
def test_steps_in_a_graph(kind):
    """append + attend captured once, replayed as lengths grow, with eager work between; the prefix's count may change."""
    H, G, D, page, b, steps = 8, 2, 64, 16, 12, 5
    f = attention.rope_frequencies(D)[0]
    g = gen(5)
    xs = [normal(g, b, H + 2 * G, D, dtype=BF).to(DEV) for _ in range(steps)]

    def fresh():
        bench = View(b, G, D, page, 1600, I8, seed=1)
        bench.append([1400 + 3 * i for i in range(b)])
        return bench

    eager, cap = fresh(), fresh()
    count = ints([80])
    kw = [dict(window=200, sinks=20) if kind == "sinks" else
          dict(prefix=attention.SharedPrefix(x.pages[:1, :85].contiguous(), count)) for x in (eager, cap)]
    kv_e, kv_c = eager.kv_len(), cap.kv_len()
    x = xs[0].clone()

    def step(bench, kv, x, how):
        kv.add_(1)
        q = bench.cache.append(x[:, H:H + G], x[:, H + G:], kv, bench.pages, q=x[:, :H], inv_freq=f)
        return bench.cache.attend(q, kv, bench.pages, **how)

    keep = [t.clone() for t in (cap.cache.k.view(I8), cap.cache.v.view(I8), cap.cache.k_scale, cap.cache.v_scale, kv_c)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap, kv_c, x, kw[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cap, kv_c, x, kw[1])
    for t, o in zip((cap.cache.k.view(I8), cap.cache.v.view(I8), cap.cache.k_scale, cap.cache.v_scale, kv_c), keep):
        t.copy_(o)
    for j in range(steps):
        x.copy_(xs[j])
        if j == 3:
            count.fill_(40)
        graph.replay()
        want = step(eager, kv_e, xs[j], kw[0])
        torch.cuda.synchronize()
        assert torch.equal(out, want), j
        torch.randn(1000, device=DEV).sum()


@pytest.mark.parametrize("kind", ["sinks", "prefix"])
def test_same_bits_on_other_streams_at_once(kind):
    b = bench_of(2, 128, 64, I8, [1900, 1700, 2000, 1800] * 6)
    q = normal(b.g, 24, 8, 128, dtype=BF).to(DEV)
    kw = dict(window=300, sinks=9) if kind == "sinks" else dict(prefix=attention.SharedPrefix(b.pages[:1, :26].contiguous(), ints([26])))
    kv = b.kv_len()
    first = b.cache.attend(q, kv, b.pages, **kw)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    many = [b.cache.attend(q, kv, b.pages, stream=s, **kw) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for x in many:
        assert torch.equal(x, first)


def test_refusals():
    b = bench_of(1, 64, 16, I8, [40, 30])
    q = normal(b.g, 2, 2, 64, dtype=BF).to(DEV)
    kv = b.kv_len()
    for kw in (dict(sinks=-1), dict(window=5, sinks=2, causal=False), dict(window=-1, sinks=2)):
        with pytest.raises(attention.binding.M3Error):
            b.cache.attend(q, kv, b.pages, **kw)
    t, c = ints([[0, 1], [2, 3]]), ints([1, 1])
    for args in ((t, c), (t.long(), c, ints([0, 1, 2])), (t, c[:1], ints([0, 1, 2])), (t, c, ints([0, 1])), (t[0], c[:1]),
                 (t.t(), c, ints([0, 1, 2])), (t.cpu(), c.cpu())):
        with pytest.raises((ValueError, TypeError)):
            attention.SharedPrefix(*args)
