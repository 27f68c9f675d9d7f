"""Calls whose launches pass 2^24 workgroups (2^32 threads): one long prompt in a large batch, many heads or sequences.
Launches of 2^32 threads along one dimension are not possible, so these go on along another."""
import math

import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests import attn_ref as ref
from tests.test_gpu_attention import BF, DEV, F32, I8, gen, normal, within

pytestmark = pytest.mark.gpu


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def test_a_long_prompt_in_a_large_batch():
    """2047 single tokens, then a prompt of 131072: with the longest for every sequence 2^24 + 2^11 workgroups of append,
    2^24 of attend. The prompt and single tokens are checked at both ends; keys 64 back are seen."""
    b, L, H, D, page, window = 2048, 131072, 8, 16, 1024, 64
    g = gen(1)
    T = b - 1 + L
    cu = torch.cat([torch.arange(b), torch.tensor([T])]).to(torch.int32).to(DEV)
    kv = torch.tensor([1] * (b - 1) + [L], dtype=torch.int32, device=DEV)
    pages = torch.full((b, L // page), -1, dtype=torch.int32)
    pages[:-1, 0] = torch.arange(b - 1, dtype=torch.int32)
    pages[-1] = torch.arange(b - 1, b - 1 + L // page, dtype=torch.int32)
    pages = pages.to(DEV)
    cache = attention.KVCache.empty(b - 1 + L // page, page, 1, D)
    k, v = normal(g, T, 1, D, dtype=BF), normal(g, T, 1, D, dtype=BF)
    q = normal(g, T, H, D, dtype=BF)
    cache.append(k.to(DEV), v.to(DEV), kv, pages, cu_q=cu, max_q=L)
    out = cache.attend(q.to(DEV), kv, pages, cu_q=cu, max_q=L, max_kv=L, window=window)
    # single tokens: one key, so its value
    one, some = (cache.read(torch.zeros(b - 1, dtype=torch.int32, device=DEV), kv[:-1], pages[:-1], 1, dtype=F32)[j].cpu()
                 for j in (1, 0))
    assert (one[:, 0] - v[:b - 1].float()).abs().max() <= 0.5 / 127 * v.float().abs().max() * 1.01
    assert (some[:, 0] - k[:b - 1].float()).abs().max() <= 0.5 / 127 * k.float().abs().max() * 1.01
    want = one[:, 0].expand(-1, H, -1).double()
    within(out[:b - 1], want, want.abs() * 2.0 ** -7 + 1e-30, "single tokens")
    for lo in (0, L // 2, L - 200):
        n = 200
        first = max(0, lo - window)
        kd, vd = (x[0].cpu() for x in cache.read(ints(first), ints(lo + n - first), pages[-1:], lo + n - first, dtype=F32))
        assert (kd - k[b - 1 + first:b - 1 + lo + n].float()).abs().max() <= 0.5 / 127 * k.float().abs().max() * 1.01
        o, _, mag, top = ref.attend(q[b - 1 + lo:b - 1 + lo + n], torch.arange(lo - first, lo - first + n), kd, vd,
                                    1 / math.sqrt(D), True, window)
        within(out[b - 1 + lo:b - 1 + lo + n], o, ref.attend_bound(o, mag, top, D, window, BF), f"prompt from {lo}")


def test_many_heads_of_many_sequences():
    """65537 sequences of 256 key heads, most slots idle: 2^24 + 2^8 workgroups of the kernel for few rows."""
    b, H, D = 65537, 256, 16
    g = gen(2)
    cache = attention.KVCache.empty(3, 16, H, D)
    kv = torch.zeros(b, dtype=torch.int32, device=DEV)
    pages = torch.zeros(b, 1, dtype=torch.int32, device=DEV)
    live = [0, 65535, 65536]
    for j, i in enumerate(live):
        kv[i], pages[i, 0] = 5 + j, j
    k, v = normal(g, 18, H, D), normal(g, 18, H, D)
    at = 0
    for i in live:
        n = int(kv[i])
        cache.append(k[at:at + n].to(DEV), v[at:at + n].to(DEV), kv[i:i + 1], pages[i:i + 1], cu_q=ints(0, n), max_q=n)
        at += n
    q = torch.zeros(b, H, D, dtype=BF, device=DEV)
    rows = normal(g, 3, H, D, dtype=BF)
    q[live] = rows.to(DEV)
    out = cache.attend(q, kv, pages, max_kv=16)
    for j, i in enumerate(live):
        n = int(kv[i])
        kd, vd = (x[0].cpu() for x in cache.read(ints(0), ints(n), pages[i:i + 1], n, dtype=F32))
        o, _, mag, top = ref.attend(rows[j:j + 1], torch.tensor([n - 1]), kd, vd, 1 / math.sqrt(D))
        within(out[i:i + 1], o, ref.attend_bound(o, mag, top, D, n, BF), f"sequence {i}")
        out[i] = 0
    assert not out.any()


def test_read_of_many_sequences():
    """2^24 + 3 sequences, one token of each."""
    b, D = (1 << 24) + 3, 16
    cache = attention.KVCache.empty(2, 16, 1, D)
    x = normal(gen(3), 2, 1, D)
    cache.append(x.to(DEV), x.to(DEV), ints(1, 1), ints(0, 1).view(2, 1))
    count = torch.zeros(b, dtype=torch.int32, device=DEV)
    pages = torch.zeros(b, 1, dtype=torch.int32, device=DEV)
    live = [0, b - 4, b - 3, b - 1]
    count[live] = 1
    pages[[live[1], live[3]]] = 1
    k, v = cache.read(torch.zeros_like(count), count, pages, 1)
    want = cache.read(ints(0, 0), ints(1, 1), ints(0, 1).view(2, 1), 1)
    for got, w in ((k, want[0]), (v, want[1])):
        assert torch.equal(got[live], w[[0, 1, 0, 1]])
        got[live] = 0
        assert not got.any()
