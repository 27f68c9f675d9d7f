"""Attention over the 8-bit cache where its arithmetic is hardest: values of any size, keys that take nearly all of the
softmax, sums that cancel; against 64 bits, with bounds that scale with the values."""
import math

import pytest
import torch

from tests import attn_ref as ref
from tests.test_gpu_attention import BF, DEV, F32, F8, I8, Bench, gen, normal, within

pytestmark = pytest.mark.gpu


def bound_of(out, mag, e, keys, v, pmax, io):
    """How far an entry may be off. e: error of a score (a probability then moves by 4 e, the sum it is divided by
    included). fp32 rows: 2^-23 of the output and of sum p |v|. bf16 rows: the output's rounding (8 significant bits:
    2^-8), each probability's to fp16 (11 bits: 2^-11, or half of fp16's least step 2^-24 in a unit of which the
    largest p * scale is at least 2^7: 2^-32 of the largest, times |code| <= |v| / scale, per key). 2^-133: bf16's
    least number."""
    r, rp = (2.0 ** -8, 2.0 ** -11) if io == BF else (2.0 ** -23, 2.0 ** -23)
    least = keys * 2.0 ** -32 * pmax[..., None] * v.double().abs().max().item() if io == BF else 0.0
    return r * out.abs() + mag * (rp * (1 + r) + 4 * e) + least + 2.0 ** -133


def against_64_bits(bench, q, n, io, scale, score_roundings, cu=None):
    """Outputs and lse of the cache's attention, each sequence's last n rows, against the values that it holds."""
    out, lse = bench.cache.attend(q.to(DEV), bench.kv_len(), bench.pages, cu_q=cu, max_q=max(n), scale=scale, lse=True)
    kd, vd = (x.cpu() for x in bench.held())
    at = 0
    for i, (c, L) in enumerate(zip(n, bench.len)):
        k, v = kd[i, :L], vd[i, :L]
        pos = torch.arange(L - c, L)
        o, z, mag, top = ref.attend(q[at:at + c], pos, k, v, scale)
        # sum p (over keys of values 1, the largest p in turn) is not needed to the bit: 1 bounds it
        pmax = torch.ones_like(z)
        e = 2.0 ** -24 * (L + score_roundings * top[..., None] + 8)
        within(out[at:at + c], o, bound_of(o, mag, e, L, v, pmax, io), f"out {i}")
        zb = e[..., 0] * 2 + z.abs() * 2.0 ** -22 + 1e-6
        g = lse[at:at + c].cpu().double()
        assert torch.isfinite(g).all() and ((g - z).abs() <= zb).all(), (i, (g - z).abs().max())
        at += c
    return out


SIZES = {  # value magnitudes by token, in turn
    "1e-33": [1e-33], "1e-35": [1e-35], "1e-33, 1": [1e-33, 1.0], "1, 1e-33": [1.0, 1e-33], "1e-30, 1e-33": [1e-30, 1e-33],
    "1e-20, 1e-33, 1": [1e-20, 1e-33, 1.0], "1e35": [1e35], "1, 1e30": [1.0, 1e30], "1e25, 1e-10": [1e25, 1e-10],
}


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt,dim", [(I8, 64), (F8, 128), (I8, 256), (F8, 64)], ids=["int8-64", "e4m3-128", "int8-256", "e4m3-64"])
@pytest.mark.parametrize("rows", [1, 70, 150])
@pytest.mark.parametrize("sizes", SIZES)
def test_values_of_any_size(sizes, rows, fmt, dim, io):
    """The softmax and its lse do not depend on how large the values are, and tiny values are not lost among themselves.
    (Lengths that are split over workgroups and joined, and that are not.)"""
    lens = [1100, 200, 33]
    n = [min(rows, L) for L in lens]
    bench = Bench(3, 1, dim, 16, max(lens), fmt, seed=dim + rows)
    T = sum(lens)
    pick = torch.cat([torch.arange(L) * len(SIZES[sizes]) // L for L in lens])
    size = torch.tensor(SIZES[sizes], dtype=torch.float64)[pick][:, None, None]
    k = normal(bench.g, T, 1, dim)
    v = (normal(bench.g, T, 1, dim).double() * size).float()
    bench.append(lens, rows=(k, v))
    q = normal(bench.g, sum(n), 2, dim, dtype=io)
    cu = None if n == [1, 1, 1] else torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32, device=DEV)
    against_64_bits(bench, q, n, io, dim ** -0.5, dim + 4, cu)


def test_a_scale_of_zero_holds_zeros_whatever_its_codes():
    """Blocks whose scale is 0 (or below the normal numbers) are zeros, also where codes are not."""
    for rows in (1, 70):
        bench = Bench(1, 1, 64, 16, 200, I8, seed=rows)
        bench.append([200])
        p = int(bench.pages[0, 2])
        bench.cache.v_scale[p] = 0.0
        bench.cache.v_scale[int(bench.pages[0, 5])] = 1e-40
        q = normal(bench.g, rows, 2, 64, dtype=F32)
        cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        out, lse = bench.cache.attend(q.to(DEV), bench.kv_len(), bench.pages, cu_q=cu, max_q=rows, lse=True)
        kd, vd = (x[0].cpu() for x in bench.held())
        vd[80:96] = 0
        assert (vd[32:48] == 0).all()
        o, z, mag, top = ref.attend(q, torch.arange(200 - rows, 200), kd, vd, 1 / 8)
        within(out, o, ref.attend_bound(o, mag, top, 64, 200, F32), "out")
        assert ((lse.cpu() - z).abs() <= 1e-4).all()


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("nats", [0, 6, 10, 14, 18, 24, 40])
@pytest.mark.parametrize("rows,dim,fmt", [(1, 64, I8), (20, 16, F8), (1, 256, F8), (70, 64, I8), (70, 128, F8), (70, 256, I8)])
def test_a_sink_with_no_value(rows, dim, fmt, nats, io):
    """The first key takes nearly all of the softmax and has no value: the output is the other keys', each of a small
    probability. Scores come from one entry (a product without rounding), so that only the softmax is in question:
    a score is rounded by the two scales, their product and the sum with the exponent (6 roundings)."""
    L = 128
    bench = Bench(1, 1, dim, 16, L, fmt, seed=dim + nats)
    k, v = torch.zeros(L, 1, dim), normal(bench.g, L, 1, dim)
    k[16:, 0, 0] = 0.5 * normal(bench.g, L - 16)
    k[0, 0, 0] = nats
    v[0] = 0.0
    k[1:16] = 0.0
    bench.append([L], rows=(k, v))
    q = torch.zeros(rows, 2, dim, dtype=io)
    q[..., 0] = 1.0
    cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    against_64_bits(bench, q, [rows], io, 1.0, 6, cu)


@pytest.mark.parametrize("dim,rows,fmt", [(64, 1, F8), (64, 3, I8), (128, 70, I8), (64, 70, F8), (256, 70, I8), (256, 2, F8)])
def test_probabilities_of_bf16_rows_keep_11_bits(dim, rows, fmt):
    """Values of both signs that cancel, a few keys: what is left shows the rounding of each probability."""
    lens = [rows + 1 + j % 5 for j in range(48)]
    bench = Bench(48, 1, dim, 16, max(lens), fmt, seed=dim + rows)
    T = sum(lens)
    v = torch.where(torch.arange(T) % 2 == 0, 1.0, -1.0)[:, None, None].expand(T, 1, dim).contiguous()
    bench.append(lens, rows=(normal(bench.g, T, 1, dim), v))
    n = [rows] * 48
    q = normal(bench.g, sum(n), 4, dim, dtype=BF)
    cu = torch.arange(0, 48 * rows + 1, rows, dtype=torch.int32, device=DEV)
    against_64_bits(bench, q, n, BF, 2.0 * dim ** -0.5, dim + 4, cu)


@pytest.mark.parametrize("lens,n", [([700, 300, 1500], [1, 1, 1]), ([900, 70, 400], [200, 70, 1]), ([2000, 40], [5, 5])], ids=str)
def test_alone_or_in_a_batch(lens, n):
    """A sequence alone and among others: the same values; their last bits may differ, as the keys may be cut elsewhere."""
    H, D = 4, 128
    bench = Bench(len(lens), 2, D, 64, max(lens), I8, seed=sum(lens))
    bench.append(list(lens))
    q = normal(bench.g, sum(n), H, D, dtype=F32).to(DEV)
    cu = torch.tensor([sum(n[:j]) for j in range(len(n) + 1)], dtype=torch.int32, device=DEV)
    whole = bench.cache.attend(q, bench.kv_len(), bench.pages, cu_q=cu, max_q=max(n))
    kd, vd = (x.cpu() for x in bench.held())
    at = 0
    for i, c in enumerate(n):
        one = bench.cache.attend(q[at:at + c], bench.kv_len()[i:i + 1], bench.pages[i:i + 1],
                                 cu_q=torch.tensor([0, c], dtype=torch.int32, device=DEV), max_q=c)
        o, _, mag, top = ref.attend(q[at:at + c].cpu(), torch.arange(lens[i] - c, lens[i]), kd[i, :lens[i]], vd[i, :lens[i]],
                                    D ** -0.5)
        bound = ref.attend_bound(o, mag, top, D, lens[i], F32)
        within(whole[at:at + c], o, bound, f"among others {i}")
        within(one, o, bound, f"alone {i}")
        at += c
