"""Values that are not finite, and memory as it may be found, where a view or a part does not look: they reach the rows
that see them and no others."""
import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests import attn_ref as ref
from tests.test_gpu_attention import BF, DEV, F32, F8, I8, normal, within
from tests.test_gpu_attention_parts import FORMS, bench, launched
from tests.test_gpu_attention_view import bench_of, ints, reference, visible

pytestmark = pytest.mark.gpu

NAN = float("nan")


def spoil(b, i, block, k_head=None, v_head=None):
    """Sequence i's block of 16 tokens as one that was given a NaN: codes as they may be, its scale NaN."""
    page, at = int(b.pages[i, block * 16 // b.page]), block % (b.page // 16)
    if k_head is not None:
        b.cache.k_scale[page, k_head, at] = NAN
    if v_head is not None:
        b.cache.v_scale[page, v_head, at] = NAN


def held_of(b):
    return [x.cpu() for x in b.held()]


def used_memory(n=1 << 22):
    """What a workspace may come out of: torch's free blocks, full of NaN."""
    for size in (n, n // 4, n // 16, n // 64):
        torch.full((size,), NAN, device=DEV)


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [I8, F8], ids=["int8", "fp8"])
@pytest.mark.parametrize("rows", [1, 20, 150])
@pytest.mark.parametrize("window,sinks", [(64, 20), (64, 0), (0, 0)])
def test_blocks_behind_a_window(rows, fmt, io, window, sinks):
    """Block 2 lies in the tile of the first tokens, blocks 15 (K, head 0) and 20 (V, head 1) inside some rows' windows."""
    D, L = 64, 430
    b = bench_of(2, D, 16, fmt, [L, 300])
    kd, vd = held_of(b)
    n = [rows, rows]
    q = normal(b.g, sum(n), 4, D, dtype=io)
    bad = [(15, 0, None), (20, None, 1)] + ([(2, 0, 1)] if window else [])
    for block, k_head, v_head in bad:
        spoil(b, 0, block, k_head, v_head)
    cu = None if rows == 1 else ints([0, rows, 2 * rows])
    used_memory()
    out = b.cache.attend(q.to(DEV), b.kv_len(), b.pages, cu_q=cu, max_q=rows, window=window, sinks=sinks)
    for i, l in enumerate(b.len):
        pos = torch.arange(l - rows, l)
        ok = visible(pos, l, True, window, sinks)
        mine = q[i * rows:(i + 1) * rows]
        o, _, mag, top = reference(mine, kd[i, :l], vd[i, :l], D ** -0.5, ok)
        hit = torch.zeros(rows, 4, dtype=torch.bool)
        if i == 0:
            for block, k_head, v_head in bad:
                sees = ok[:, 16 * block:16 * block + 16].any(1)
                for head in (k_head, v_head):
                    if head is not None:
                        hit[:, 2 * head:2 * head + 2] |= sees[:, None]
        got = out[i * rows:(i + 1) * rows].cpu()
        assert got[hit].isnan().all(), i
        bound = ref.attend_bound(o, mag, top, D, l, io)
        within(got[~hit], o[~hit], bound[~hit], f"out {i}")


@pytest.mark.parametrize("fmt", [I8, F8], ids=["int8", "fp8"])
@pytest.mark.parametrize("form,batch,H,kv", [("items", 16, 8, 2), ("join", 130, 16, 4), ("merge", 60, 64, 8)])
def test_rows_that_share_a_prefix(form, batch, H, kv, fmt):
    """A sequence's own spoiled keys and another's spoiled query stay theirs, though their rows share tiles; a spoiled
    prefix reaches its group, for the key head that holds it."""
    page, D = 16, 64
    starts, counts = [0, batch // 2, batch], [20, 31]
    lens = [counts[i >= batch // 2] * page + 20 + i % 40 for i in range(batch)]
    b = bench(batch, kv, D, page, fmt, lens, seed=6)
    q = normal(b.g, batch, H, D, dtype=BF)
    q[4, 1] = NAN
    spoil(b, 7, counts[0], k_head=0)
    spoil(b, batch - 3, counts[1], v_head=1)
    sample = {0, 3, 5, 6, 8, batch // 2 - 1, batch // 2, batch - 4, batch - 2} - {4, 7, batch - 3}
    G = H // kv
    used_memory()
    out, names = launched(lambda: b.run(q, [1] * batch, BF, starts, counts, room=8192, sample=sample))
    assert not names or tuple(names) == FORMS[form], names
    bad = out.isnan().any(-1).cpu()
    want = torch.zeros(batch, H, dtype=torch.bool)
    want[4, 1] = True
    want[7, :G] = True
    want[batch - 3, G:2 * G] = True
    assert torch.equal(bad, want)
    donor = max(range(batch // 2), key=lambda i: lens[i])
    spoil(b, donor, 3, v_head=1)
    used_memory()
    out = b.run(q, [1] * batch, BF, starts, counts, room=8192, sample={i for i in sample if i >= batch // 2})
    want[:batch // 2, G:2 * G] = True
    assert torch.equal(out.isnan().any(-1).cpu(), want)


def test_the_prefix_of_one_pass():
    """The same where every sequence reads the prefix itself."""
    D, page = 64, 16
    for rows in (1, 40):
        b = bench_of(2, D, page, F8, [300, 280, 290, 270])
        kd, vd = held_of(b)
        spoil(b, 1, 16, k_head=0)
        shared = ints([b.pages[0, :12].tolist(), b.pages[2, :12].tolist()])
        q = normal(b.g, 4 * rows, 4, D, dtype=BF)
        q[3 * rows, 3] = NAN
        spoil(b, 2, 5, v_head=0)
        used_memory()
        out = b.cache.attend(q.to(DEV), b.kv_len(), b.pages, cu_q=None if rows == 1 else ints([rows * i for i in range(5)]),
                             max_q=rows, prefix=attention.SharedPrefix(shared, ints([12, 12]), ints([0, 2, 4])))
        bad = out.isnan().any(-1).cpu().view(4, rows, 4)
        want = torch.zeros_like(bad)
        want[2:, :, :2] = True
        want[3, 0, 3] = True
        seen = torch.arange(280 - rows, 280) >= 256
        want[1, seen, :2] = True
        assert torch.equal(bad, want)
        for i, donor in ((0, 0), (1, 0), (2, 2), (3, 2)):
            l = b.len[i]
            k, v = (torch.cat([x[donor, :192], x[i, 192:l]]) for x in (kd, vd))
            o, _, mag, top = reference(q[i * rows:(i + 1) * rows].nan_to_num(0.0), k, v, D ** -0.5,
                                       visible(torch.arange(l - rows, l), l, True, 0, 0))
            keep = ~want[i]
            within(out[i * rows:(i + 1) * rows].cpu()[keep], o[keep], ref.attend_bound(o, mag, top, D, l, BF)[keep], f"out {i}")


@pytest.mark.parametrize("wide", [2047, 2048, 4096])
def test_prefix_tables_wider_than_positions(wide):
    """Pages of 2^20 tokens: a table may name more than 2^31 tokens' worth; its rows lie where they are."""
    D, page = 16, 1 << 20
    c = attention.KVCache.empty(3, page, 1, D, dtype=I8)
    g = torch.Generator().manual_seed(wide)
    k, v = torch.randn(150, 1, D, generator=g), torch.randn(150, 1, D, generator=g)
    own = ints([[0], [1], [-1]])
    c.append(k.to(DEV), v.to(DEV), ints([60, 90]), own[:2].contiguous(), cu_q=ints([0, 60, 150]), max_q=90)
    table = torch.full((2, wide), -1, dtype=torch.int32, device=DEV)
    table[0, 0], table[1, 0] = 0, 1
    q = torch.randn(3, 2, D, generator=g).to(DEV)
    lens = ints([60, 90, 80])
    got = c.attend(q, lens, torch.full_like(own, -1), prefix=attention.SharedPrefix(table, ints([1, 1]), ints([0, 1, 3])))
    want = c.attend(q, lens, ints([[0], [1], [1]]))
    assert want.abs().amin(-1).max() > 0 and (got - want).abs().max() <= 2.0 ** -18 * want.abs().max()
