"""Calls whose bound on the rows, `max_q`, is left out or too small: every row that is kept has its own position."""
import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests import attn_ref as ref
from tests.test_gpu_attention import BF, DEV, F32, I8, F8, Bench, gen, normal, turn_bound, within

pytestmark = pytest.mark.gpu


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def held(cache, kv, pages, top):
    return cache.read(torch.zeros_like(kv), kv, pages, top, dtype=F32)


@pytest.mark.parametrize("n", [[20], [37, 0, 5], [1, 300]], ids=str)
def test_without_max_q(n):
    """The row count bounds every sequence: append and attend give what they give with the longest named."""
    H, G, D = 4, 2, 64
    g = gen(sum(n))
    T, b = sum(n), len(n)
    k, v, q = (normal(g, T, h, D, dtype=BF).to(DEV) for h in (G, G, H))
    f = attention.rope_frequencies(D)[0]
    cu = ints(*[sum(n[:j]) for j in range(b + 1)])
    kv = ints(*n)
    benches = [Bench(b, G, D, 16, max(n), I8), Bench(b, G, D, 16, max(n), I8)]
    got = []
    for bench, bound in zip(benches, ({}, dict(max_q=max(n)))):
        t = bench.cache.append(k, v, kv, bench.pages, cu_q=cu, q=q, inv_freq=f, **bound)
        got.append((t, *held(bench.cache, kv, bench.pages, max(n))))
        want = ref.turn(q.cpu(), torch.cat([torch.arange(c) for c in n]), f.cpu())
        within(t, want, turn_bound(q.cpu(), want, 1.0, BF), "q")
    for a, b2 in zip(*got):
        assert torch.equal(a, b2)
    bench = benches[0]
    bench.len = list(n)
    out = bench.cache.attend(q, kv, bench.pages, cu_q=cu)
    kd, vd = got[0][1].cpu(), got[0][2].cpu()
    at = 0
    for i, c in enumerate(n):
        o, _, mag, top = ref.attend(q[at:at + c].cpu(), torch.arange(c), kd[i, :c], vd[i, :c], D ** -0.5)
        within(out[at:at + c], o, ref.attend_bound(o, mag, top, D, c, BF), f"out {i}")
        at += c


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("before,n,most", [(0, 20, 5), (21, 40, 17), (7, 3, 1), (30, 200, 130)])
def test_append_of_more_rows_than_max_q(before, n, most, io):
    """The first max_q rows are stored and turned at their own positions, the others are left out."""
    G, D, H = 2, 64, 3
    f = attention.rope_frequencies(D, device="cpu")[0]
    bench = Bench(1, G, D, 16, before + n, F8, seed=n)
    bench.append([before], inv_freq=f)
    k, v, q = (normal(bench.g, n, h, D, dtype=io) for h in (G, G, H))
    pos = torch.arange(before, before + n)
    bench.ref.append(0, before, ref.turn(k, pos, f)[:most].float(), v[:most])
    out = torch.zeros(n, H, D, dtype=io, device=DEV)
    bench.cache.append(k.to(DEV), v.to(DEV), ints(before + n), bench.pages, cu_q=ints(0, n), max_q=most, q=q.to(DEV),
                       q_out=out, inv_freq=f.to(DEV))
    want = ref.turn(q, pos, f)
    want[most:] = 0
    within(out, want, turn_bound(q, want, 1.0, io), "q")
    bench.len = [before + most]
    bench.check(times=2, rare=io == F32)


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 9), (False, 0)])
@pytest.mark.parametrize("lens,n,most", [([50, 33], [20, 3], 4), ([300, 260], [200, 150], 130)])
def test_attend_of_more_rows_than_max_q(lens, n, most, causal, window, io):
    """The first max_q rows of a sequence see the keys of their own positions; the others are left as they were."""
    G, D, H = 2, 64, 4
    bench = Bench(2, G, D, 16, max(lens), I8, seed=most)
    bench.append(list(lens))
    q = normal(bench.g, sum(n), H, D, dtype=io)
    out = torch.full((sum(n), H, D), 7.0, dtype=io, device=DEV)
    bench.cache.attend(q.to(DEV), ints(*lens), bench.pages, cu_q=ints(0, n[0], sum(n)), max_q=most, causal=causal,
                       window=window, out=out)
    kd, vd = (x.cpu() for x in bench.held())
    at = 0
    for i, c in enumerate(n):
        keep = min(c, most)
        o, _, mag, top = ref.attend(q[at:at + keep], torch.arange(lens[i] - c, lens[i] - c + keep), kd[i, :lens[i]],
                                    vd[i, :lens[i]], D ** -0.5, causal, window)
        within(out[at:at + keep], o, ref.attend_bound(o, mag, top, D, lens[i], io), f"out {i}")
        assert (out[at + keep:at + c] == 7.0).all()
        at += c
