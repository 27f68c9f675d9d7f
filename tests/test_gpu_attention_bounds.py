"""Bounds that are too large size the launch only: pieces of prompts and prompts under loose `max_kv` (the page table's
room is the default) and `max_q` see the same keys, and their keys are cut by what each row tile sees, so that a call
under a loose bound has the bits of the tight one wherever both have as many workgroups."""
import pytest
import torch

from tests import attn_ref as ref
from tests.test_gpu_attention import BF, DEV, F32, F8, I8, Bench, normal, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kv,H,dim,fmt,lens,n,window", [
    (1, 4, 64, I8, [4000], [100], 0), (1, 4, 128, F8, [4100, 1500], [80, 70], 0), (2, 2, 256, I8, [2000], [70], 0),
    (1, 4, 64, F8, [5000], [90], 1700), (1, 2, 128, I8, [700], [700], 0), (1, 8, 64, I8, [130, 2500, 0, 600], [130, 64, 1, 9], 0)])
def test_loose_bounds(kv, H, dim, fmt, lens, n, window, io):
    bench = Bench(len(lens), kv, dim, 64, 20000, fmt, seed=dim)
    bench.append(list(lens))
    q = normal(bench.g, sum(n), H, dim, dtype=io)
    cu = torch.tensor([sum(n[:j]) for j in range(len(n) + 1)], dtype=torch.int32, device=DEV)
    kd, vd = (x.cpu() for x in bench.held())
    outs = []
    for max_kv, max_q in ((max(lens), max(n)), (8192, max(n)), (None, max(n)), (None, None)):
        out, lse = bench.cache.attend(q.to(DEV), bench.kv_len(), bench.pages, cu_q=cu, max_q=max_q, max_kv=max_kv,
                                      window=window, lse=True)
        at = 0
        for i, (c, L) in enumerate(zip(n, lens)):
            o, z, mag, top = ref.attend(q[at:at + c], torch.arange(L - c, L), kd[i, :L], vd[i, :L], dim ** -0.5, True, window)
            within(out[at:at + c], o, ref.attend_bound(o, mag, top, dim, L, io), f"out {i}")
            g = lse[at:at + c].cpu().double()
            zb = 2.0 ** -24 * (L + (dim + 4) * top + 8) * 2 + z.abs() * 2.0 ** -22 + 1e-6
            assert torch.equal(torch.isinf(g), torch.isinf(z)) and (((g - z).abs() <= zb) | torch.isinf(z)).all()
            at += c
        outs.append(out)
    assert torch.equal(outs[1], outs[2])


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
def test_a_piece_is_cut_as_under_the_tight_bound(io):
    """512 rows that end at 8192, under its own bound and one of 131072: as many workgroups, so the same cuts."""
    bench = Bench(1, 1, 64, 64, 131072, I8, seed=5)
    bench.append([8192])
    q = normal(bench.g, 512, 4, 64, dtype=io).to(DEV)
    cu = torch.tensor([0, 512], dtype=torch.int32, device=DEV)
    a, b, c = (bench.cache.attend(q, bench.kv_len(), bench.pages, cu_q=cu, max_q=512, max_kv=m) for m in (8192, 40000, None))
    assert torch.equal(a, b) and torch.equal(a, c)
