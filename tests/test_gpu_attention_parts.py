"""Prefixes computed as parts of their own (many sequences for a group's pages), each way the plan takes, against 64 bits:
the prefix among the items of the launch for few rows; in a launch of the kernel for many rows, joined by the sequences'
own workgroups, or by the merge. The plan goes by bounds, so a wide table with short prefixes takes these ways too."""
import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests.test_gpu_attention import BF, DEV, F32, F8, I8, gen, normal
from tests.test_gpu_attention_view import View, ints, reference, visible
from tests import attn_ref as ref
from tests.test_gpu_attention import within

pytestmark = pytest.mark.gpu

# which way a call takes is told by its launches
FORMS = {"items": ("attend_rows", "attend_merge"), "join": ("attend_tile", "attend_rows"),
         "merge": ("attend_tile", "attend_rows", "attend_merge")}


def launched(fn):
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        out = fn()
        torch.cuda.synchronize()
    names = [e.name for e in sorted(p.events(), key=lambda e: e.time_range.start)]
    return out, [k for n in names for k in ("attend_rows", "attend_tile", "attend_merge", "attend_join") if k + "_kernel" in n]


class Parts(View):
    """A prefix table as wide as `room`, page tables too: what the plan sees are those bounds."""

    def run(self, q, n, io, starts, counts, lens=None, room=4096, causal=True, cu=None, form=None, sample=None, max_kv=None):
        lens = self.len if lens is None else lens
        wide = room // self.page
        shared = torch.full((len(counts), wide), -7, dtype=torch.int32, device=DEV)
        pages = torch.full((self.batch, wide), -3, dtype=torch.int32, device=DEV)
        pages[:, :self.pages.shape[1]] = self.pages
        first = [(None, 0)] * self.batch
        for g, c in enumerate(counts):
            members = range(starts[g], starts[g + 1])
            if not members:
                continue
            donor = max(members, key=lambda i: self.len[i])
            shared[g, :c] = self.pages[donor, :c]
            for i in members:
                first[i] = (donor, c * self.page)
                pages[i, :c] = self.spare[0].item() if i % 2 else -3
        prefix = attention.SharedPrefix(shared, ints(counts), None if starts == [0, self.batch] else ints(starts))
        if cu is None and n != [1] * self.batch:
            cu = ints([sum(n[:j]) for j in range(len(n) + 1)])
        call = lambda: self.cache.attend(q.to(DEV), ints(lens), pages, cu_q=cu, causal=causal, prefix=prefix,  # noqa: E731
                                         max_q=max(n + [1]), max_kv=max_kv, lse=True)
        out, lse = call()
        if form is not None:
            again, names = launched(call)
            assert not names or tuple(names) == FORMS[form], names          # (none: the profiler sees no launches here)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)
        kd, vd = (x.cpu() for x in self.held())
        at = 0
        for i, c in enumerate(n):
            L, (d, p) = lens[i], first[i]
            p = min(p, L)
            if sample is None or i in sample:
                k = torch.cat([kd[d, :p], kd[i, p:L]]) if p else kd[i, :L]
                v = torch.cat([vd[d, :p], vd[i, p:L]]) if p else vd[i, :L]
                pos = torch.arange(L - c, L)
                o, z, mag, top = reference(q[at:at + c].cpu(), k, v, self.dim ** -0.5, visible(pos, L, causal, 0, 0))
                within(out[at:at + c], o, ref.attend_bound(o, mag, top, self.dim, L, io), f"out {i}")
                zb = 2.0 ** -24 * (L + (self.dim + 4) * top + 8) * 2 + z.abs() * 2.0 ** -22 + 1e-6
                y = lse[at:at + c].cpu().double()
                assert torch.equal(torch.isinf(y), torch.isinf(z)) and (((y - z).abs() <= zb) | torch.isinf(z)).all(), i
            at += c
        return out


def bench(batch, kv, D, page, fmt, lens, seed=0):
    b = Parts(batch, kv, D, page, max(lens + [1]), fmt, seed=seed + D, spare=2)
    b.append(list(lens))
    return b


CASES = [  # form, kv heads, q heads, dim, page, fmt, io, batch, rows, prefix pages of each group, room, longest tail
    ("items", 4, 16, 128, 64, I8, BF, 16, 1, [9], 4096, 300),
    ("items", 2, 8, 64, 16, F8, F32, 24, 1, [30, 0, 11], 8192, 90),
    ("items", 1, 6, 80, 32, I8, BF, 30, 3, [7, 12, 2, 20], 16384, 200),
    ("items", 2, 8, 256, 64, F8, BF, 12, 1, [5], 4096, 150),
    ("items", 1, 6, 128, 16, I8, F32, 10, 1, [37], 16384, 33),
    ("items", 3, 3, 16, 16, I8, F32, 70, 2, [3, 60], 8192, 70),
    ("join", 4, 16, 128, 64, F8, BF, 140, 1, [9], 8192, 150),
    ("join", 8, 8, 64, 16, I8, F32, 80, 1, [20, 33], 8192, 60),
    ("join", 2, 2, 32, 16, F8, BF, 300, 1, [10, 3, 0, 25, 31], 4096, 40),
    ("join", 8, 64, 128, 64, I8, BF, 72, 1, [6], 4096, 100),
    ("join", 8, 64, 64, 16, F8, BF, 200, 1, [10], 4096, 50),            # 128 rows a tile
    ("join", 8, 64, 128, 64, F8, BF, 300, 1, [2], 4096, 40),            # 256
    ("join", 4, 8, 256, 32, I8, F32, 70, 1, [12], 4096, 60),
    ("join", 4, 12, 96, 16, I8, BF, 150, 2, [21, 17, 5], 4096, 60),
    ("merge", 8, 64, 64, 16, I8, BF, 60, 1, [30], 4096, 200),
    ("merge", 8, 32, 128, 32, F8, F32, 60, 1, [10, 7], 8192, 100),
    ("merge", 4, 16, 256, 64, I8, BF, 60, 1, [5], 16384, 120),
    ("merge", 2, 24, 112, 16, F8, BF, 60, 3, [33, 0, 64], 8192, 70),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_ways(case):
    """Idle slots, sequences that hold nothing of their own or end inside the prefix, rows of nothing, among the others."""
    form, kv, H, D, page, fmt, io, batch, rows, counts, room, tail = case
    g = gen(batch + D + H)
    starts = [i * batch // len(counts) for i in range(len(counts) + 1)]
    of = [max(j for j in range(len(counts)) if starts[j] <= i) for i in range(batch)]
    extra = torch.randint(1, tail, (batch,), generator=g).tolist()
    lens = [counts[of[i]] * page + extra[i] + rows - 1 for i in range(batch)]
    lens[1] = 0
    lens[2] = counts[of[2]] * page
    lens[3] = max(1, counts[of[3]] * page // 2 + 1)
    lens[-1] = max(1, counts[of[-1]] * page - 1)
    n = [1] * batch if rows == 1 else torch.randint(0, rows + 1, (batch,), generator=g).tolist()
    if rows > 1:
        n[0], n[5] = rows, 0
    b = bench(batch, kv, D, page, fmt, lens, seed=H)
    q = normal(b.g, sum(n), H, D, dtype=io)
    sample = set(range(0, batch, max(1, batch // 24))) | {1, 2, 3, batch - 1}
    b.run(q, n, io, starts, counts, room=room, form=form, sample=sample)


@pytest.mark.parametrize("form,batch,H,kv", [("items", 16, 8, 2), ("join", 130, 16, 4), ("merge", 60, 64, 8)])
def test_sequences_of_no_group_and_empty_groups(form, batch, H, kv):
    """Groups that begin late, end early, hold nobody or lie apart; without causal masks too; under a bound below lengths."""
    page, D = 16, 64
    g = gen(batch)
    starts = [3, batch // 2, batch // 2, batch - 2]
    counts = [20, 9, 31]
    lens = torch.randint(31 * page + 1, 32 * page + 150, (batch,), generator=g).tolist()
    b = bench(batch, kv, D, page, I8, lens, seed=1)
    q = normal(b.g, batch, H, D, dtype=BF)
    sample = {0, 2, 3, 4, batch // 2 - 1, batch // 2, batch - 3, batch - 2, batch - 1}
    b.run(q, [1] * batch, BF, starts, counts, room=8192, form=form, sample=sample)
    b.run(q, [1] * batch, BF, starts, counts, room=8192, causal=False, sample=sample)


@pytest.mark.parametrize("form,batch,H,kv", [("items", 16, 8, 2), ("join", 130, 16, 4), ("merge", 60, 64, 8)])
def test_rows_left_as_they_were_and_nothing_seen(form, batch, H, kv):
    """Rows behind the last sequence and past max_q keep what they held; rows that see nothing give 0 and -inf."""
    page, D = 16, 64
    b = bench(batch, kv, D, page, F8, [40 * page + 5 + i % 9 for i in range(batch)], seed=2)
    q = normal(b.g, batch + 20, H, D, dtype=F32).to(DEV)
    n = [1] * (batch - 1) + [4]
    cu = ints([sum(n[:j]) for j in range(batch + 1)])
    wide = torch.full((1, 512), -1, dtype=torch.int32, device=DEV)
    wide[0, :40] = b.pages[0, :40]
    pages = torch.full((batch, 512), -1, dtype=torch.int32, device=DEV)
    pages[:, :b.pages.shape[1]] = b.pages
    prefix = attention.SharedPrefix(wide, ints([40]))
    out = torch.full((batch + 20, H, D), 3.0, device=DEV)
    b.cache.attend(q, b.kv_len(), pages, cu_q=cu, max_q=2, prefix=prefix, out=out)
    assert (out[batch + 1:] == 3.0).all() and (out[:batch + 1] != 3.0).any(-1).any(-1).all()
    none, lse = b.cache.attend(q[:batch], torch.zeros_like(b.kv_len()), pages, prefix=prefix, lse=True)
    assert (none == 0).all() and (lse == -float("inf")).all()
    wide.fill_(-1)
    pages.fill_(-1)
    none, lse = b.cache.attend(q[:batch], b.kv_len(), pages, prefix=prefix, lse=True)
    assert (none == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("form,batch,H,kv", [("items", 16, 8, 2), ("join", 130, 16, 4), ("merge", 60, 64, 8)])
def test_graph_streams_and_arrays_out_of_range(form, batch, H, kv):
    """Captured and replayed as lengths and the count change; on three streams at once; arrays that make no sense."""
    page, D = 16, 64
    b = bench(batch, kv, D, page, I8, [40 * page + 3 + i % 30 for i in range(batch)], seed=3)
    q = normal(b.g, batch, H, D, dtype=BF).to(DEV)
    wide = torch.full((1, 512), -1, dtype=torch.int32, device=DEV)
    wide[0, :40] = b.pages[0, :40]
    pages = torch.full((batch, 512), -1, dtype=torch.int32, device=DEV)
    pages[:, :b.pages.shape[1]] = b.pages
    count, kv_len = ints([40]), b.kv_len()
    prefix = attention.SharedPrefix(wide, count)
    call = lambda **kw: b.cache.attend(q, kv_len, pages, prefix=prefix, **kw)  # noqa: E731
    first, names = launched(call)
    assert not names or tuple(names) == FORMS[form], names
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    many = [call(stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, first) for x in many)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for step, c in enumerate((40, 40, 33, 0, 12)):
        count.fill_(c)
        kv_len.sub_(step)
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(out, want), step
    for starts, counts in (([0, 99, -4], [2 ** 31 - 1, -5]), ([-2 ** 31, 2, 2 ** 31 - 1], [1, 2]), ([batch, batch, batch], [40, 40]),
                           ([3, 1, 2], [2, 512])):
        p = attention.SharedPrefix(wide.expand(2, 512).contiguous().random_(-2 ** 31, 2 ** 31 - 1), ints(counts), ints(starts))
        b.cache.attend(q, kv_len, pages, prefix=p)
        b.cache.attend(q, ints([2 ** 31 - 1, -3] * (batch // 2)), pages, prefix=p)
        cu = torch.randint(-batch, 2 * batch, (batch + 1,), generator=gen(4)).to(torch.int32).to(DEV)
        b.cache.attend(q, kv_len, pages, prefix=p, cu_q=cu, max_q=3)
    torch.cuda.synchronize()
