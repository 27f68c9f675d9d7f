"""Ragged batches under a bound on the rows that is far above most sequences (or left out): work is dealt out by the rows
that are there, one sequence's after the other's. Against 64 bits and the same call under the tight bound."""
import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests import attn_ref as ref
from tests.test_gpu_attention import BF, DEV, F32, F8, I8, Bench, gen, normal, within

pytestmark = pytest.mark.gpu


def offsets(n):
    return torch.tensor([sum(n[:j]) for j in range(len(n) + 1)], dtype=torch.int32, device=DEV)


def ragged(seed, b, top, longest, zeros=0.3):
    g = gen(seed)
    n = torch.randint(0, top + 1, (b,), generator=g)
    n[torch.rand(b, generator=g) < zeros] = 0
    n[b // 3] = longest
    return n.tolist()


@pytest.mark.parametrize("io,inter", [(BF, False), (F32, True)], ids=["bf16-half", "f32-interleaved"])
@pytest.mark.parametrize("seed,b,top,longest", [(1, 40, 3, 400), (2, 300, 1, 90), (3, 3, 0, 1000), (4, 90, 40, 700)])
def test_append(seed, b, top, longest, io, inter):
    """Codes, scales and turned queries bit for bit as under the tight bound and as each sequence by itself."""
    G, H, D = 2, 4, 64
    n = ragged(seed, b, top, longest)
    before = torch.randint(0, 40, (b,), generator=gen(seed + 50)).tolist()
    f = attention.rope_frequencies(D)[0]
    T = sum(n)
    g = gen(seed)
    k, v, q = (normal(g, T, h, D, dtype=io).to(DEV) for h in (G, G, H))
    old = normal(g, sum(before), G, D, dtype=io).to(DEV)
    lens = [x + y for x, y in zip(before, n)]
    kv, cu = torch.tensor(lens, dtype=torch.int32, device=DEV), offsets(n)
    got = []
    for how in ("tight", "loose", "none", "one by one"):
        bench = Bench(b, G, D, 16, max(lens), I8, seed=seed)
        bench.len = list(before)
        bench.cache.append(old, old, bench.kv_len(), bench.pages, cu_q=offsets(before), max_q=max(before))
        kw = dict(inv_freq=f, interleaved=inter)
        if how == "one by one":
            out, at = torch.empty_like(q), 0
            for i, c in enumerate(n):
                if c:
                    bench.cache.append(k[at:at + c], v[at:at + c], kv[i:i + 1], bench.pages[i:i + 1], cu_q=offsets([c]), max_q=c,
                                       q=q[at:at + c], q_out=out[at:at + c], **kw)
                at += c
        else:
            most = {"tight": max(n), "loose": 3 * T, "none": None}[how]
            out = bench.cache.append(k, v, kv, bench.pages, cu_q=cu, max_q=most, q=q, **kw)
        zero = torch.zeros(b, dtype=torch.int32, device=DEV)
        got.append((out, *bench.cache.read(zero, kv, bench.pages, max(lens), dtype=F32)))
    for other in got[1:]:
        for x, y in zip(got[0], other):
            assert torch.equal(x, y)


ATTEND = [  # heads, key heads, dim, format, longest context, sequences, rows up to, longest
    (4, 2, 64, I8, 300, 200, 1, 60),      # mostly single tokens: few rows, whole row tiles
    (8, 2, 128, F8, 3000, 5, 2, 9),       # few rows over long contexts: even shares
    (4, 1, 96, I8, 2500, 12, 1, 40),
    (2, 1, 256, F8, 1500, 6, 3, 12),
    (4, 2, 64, I8, 500, 30, 60, 480),     # prompts and pieces: many rows
    (8, 2, 128, F8, 1500, 4, 100, 900),
    (4, 2, 256, I8, 700, 8, 30, 500),
]


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("H,G,D,fmt,top,b,rows,longest", ATTEND)
def test_attend(H, G, D, fmt, top, b, rows, longest, window, io):
    n = ragged(b + rows, b, rows, longest, zeros=0.2)
    g = gen(D + b)
    lens = torch.randint(0, top, (b,), generator=g).tolist()
    lens[0], lens[b // 3] = top, max(longest, top // 2)
    bench = Bench(b, G, D, 16, top, fmt, seed=D)
    bench.append(lens)
    q = normal(g, sum(n), H, D, dtype=io)
    tight = bench.attend(q, n, io, window=window, max_kv=top, cu=offsets(n))
    for most in (2 * sum(n), max(n) + 100):
        loose = bench.attend(q, n, io, window=window, max_q=most, cu=offsets(n))
        assert loose.shape == tight.shape
    kv, cu = bench.kv_len(), offsets(n)
    a = bench.cache.attend(q.to(DEV), kv, bench.pages, cu_q=cu, window=window)
    assert torch.equal(a, bench.cache.attend(q.to(DEV), kv, bench.pages, cu_q=cu, window=window))


def test_offsets_that_make_no_sense_stay_in_bounds():
    """Offsets that fall, are negative or pass the rows: nothing is written outside the outputs and pages."""
    b, T, D = 9, 60, 64
    bench = Bench(b, 1, D, 16, 128, I8, seed=3)
    bench.append([100] * b)
    spare = bench.cache.k.view(I8)[bench.spare].clone()
    big = torch.full((T + 40, 4, D), 5.0, dtype=BF, device=DEV)
    q = normal(bench.g, T, 4, D, dtype=BF).to(DEV)
    kn = normal(bench.g, T, 1, D, dtype=BF).to(DEV)
    for cu in ([0, 50, 10, 10, -7, 3, 2 ** 31 - 1, -2 ** 31, 60, 5], [60] * 10, [0] * 10, [9, 8, 7, 6, 5, 4, 3, 2, 1, 0]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        for most in (1, 13, None):
            out = big[20:20 + T]
            bench.cache.attend(q, bench.kv_len(), bench.pages, cu_q=cu, max_q=most, out=out)
            bench.cache.append(kn, kn, bench.kv_len(), bench.pages, cu_q=cu, max_q=most, q=q, q_out=out)
    torch.cuda.synchronize()
    assert (big[:20] == 5.0).all() and (big[20 + T:] == 5.0).all()
    assert torch.equal(bench.cache.k.view(I8)[bench.spare], spare)
