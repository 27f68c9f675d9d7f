"""Checks of the attention layer's C entry points that need no GPU: what include/m3_attn.h declares is exported, the
plan's workspace, and every refusal before any HIP call. Pointers are fake, aligned addresses, never dereferenced."""
import ctypes
import os
import re

import pytest

from mamba_ssm_scan_amd import attention as at
from mamba_ssm_scan_amd import binding as bd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 30
FAKE = 1 << 44


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from mamba_ssm_scan_amd import build
        build.build()
    return at._lib()


def place(j):
    return FAKE + 64 * j * G


def cache(**kw):
    d = dict(k=place(0), v=place(1), k_scale=place(2), v_scale=place(3), num_pages=100, page_size=64, heads=4,
             headdim=128, format=0)
    d.update(kw)
    return at.M3KvCache(*[d[n] for n, _ in at.M3KvCache._fields_])


def batch(**kw):
    d = dict(batch=3, tokens=3, max_pages=8, max_q=1, max_kv=512, cu_q=None, kv_len=place(4), pages=place(5))
    d.update(kw)
    return at.M3KvBatch(*[d[n] for n, _ in at.M3KvBatch._fields_])


def rows(j, heads=4, dim=128, **kw):
    d = dict(p=place(j), token_stride=heads * dim, head_stride=dim)
    d.update(kw)
    return at.M3Rows(d["p"], d["token_stride"], d["head_stride"])


def rotary(**kw):
    d = dict(inv_freq=place(6), rot=128, interleaved=0, mscale=1.0)
    d.update(kw)
    return at.M3Rotary(d["inv_freq"], d["rot"], d["interleaved"], d["mscale"])


def refused(lib, status, text, code):
    assert status == code, (status, lib.m3_last_error())
    assert text in lib.m3_last_error().decode(), lib.m3_last_error()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "m3_attn.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(m3_[a-z_]+)\s*\(", src)))
    assert names == sorted(at.EXPORTS)
    for n in names:
        assert hasattr(lib, n)


def rope(lib, x=None, y=None, tokens=5, heads=4, dim=128, io=1, pos=place(9), rot=None):
    return lib.m3_rope(x or rows(7), y or rows(8), tokens, heads, dim, io, pos, rot or rotary(), 0, None)


def test_rope_refusals(lib):
    refused(lib, rope(lib, io=5), "dtype", 3)
    refused(lib, rope(lib, tokens=-1), "tokens", 1)
    refused(lib, rope(lib, heads=0), "heads", 1)
    refused(lib, rope(lib, dim=1), "headdim", 1)
    refused(lib, lib.m3_rope(None, rows(8), 5, 4, 128, 1, place(9), rotary(), 0, None), "x is NULL", 1)
    refused(lib, rope(lib, x=rows(7, p=None)), "x is NULL", 1)
    refused(lib, rope(lib, x=rows(7, p=place(7) + 1)), "x", 4)
    refused(lib, rope(lib, y=rows(8, token_stride=-4)), "y: a stride", 1)
    refused(lib, rope(lib, y=rows(8, token_stride=(1 << 31) + 1)), "y: a stride", 1)
    refused(lib, rope(lib, y=rows(8, head_stride=127)), "rows overlap", 1)
    refused(lib, rope(lib, y=rows(8, token_stride=0)), "rows overlap", 1)
    refused(lib, rope(lib, y=rows(8, token_stride=511)), "rows overlap", 1)
    refused(lib, rope(lib, pos=None), "positions", 1)
    refused(lib, rope(lib, pos=place(9) + 2), "positions", 4)
    refused(lib, lib.m3_rope(rows(7), rows(8), 5, 4, 128, 1, place(9), None, 0, None), "rotary", 1)
    for kw, code in ((dict(rot=0), 1), (dict(rot=3), 1), (dict(rot=130), 1), (dict(inv_freq=None), 1),
                     (dict(inv_freq=place(6) + 2), 4), (dict(mscale=float("nan")), 1), (dict(mscale=float("inf")), 1)):
        assert rope(lib, rot=rotary(**kw)) == code, kw
    refused(lib, rope(lib, y=rows(7, p=place(7) + 16)), "y overlaps x", 1)
    refused(lib, rope(lib, y=rows(8, p=place(9))), "y overlaps positions", 1)
    refused(lib, rope(lib, y=rows(8, p=place(6))), "y overlaps inv_freq", 1)
    # interleaved parts of one buffer: no overlap while they stay apart; the check is told by the first byte shared
    refused(lib, rope(lib, x=rows(7, token_stride=1024), y=rows(7, p=place(7) + 1022, token_stride=1024)), "y overlaps x", 1)
    assert rope(lib, tokens=0, x=rows(7, p=None), y=rows(8, p=None), pos=None) == 0


def test_cache_refusals(lib):
    def size(c, b=None, h=8, io=1, causal=1, window=0):
        return lib.m3_kv_attend(c, b or batch(), rows(10, 8), place(11), None, h, io, 1.0, causal, window, None, 0, None)
    refused(lib, size(None), "cache is NULL", 1)
    for kw, text, code in ((dict(format=2), "format", 3), (dict(num_pages=-1), "num_pages", 1),
                           (dict(page_size=8), "page_size", 1), (dict(page_size=48), "page_size", 1),
                           (dict(heads=0), "heads", 1), (dict(headdim=24), "headdim", 5), (dict(headdim=272), "headdim", 5),
                           (dict(k=None), "cache k", 1), (dict(v=place(1) + 8), "cache v", 4),
                           (dict(k_scale=None), "k_scale", 1), (dict(v_scale=place(3) + 4), "v_scale", 4),
                           (dict(num_pages=1 << 31, page_size=1 << 20), "sizes", 1)):
        refused(lib, size(cache(**kw)), text, code)
    for kw, text, code in ((dict(batch=-1), "batch", 1), (dict(tokens=4), "cu_q", 2), (dict(max_q=-1), "max_q", 1),
                           (dict(max_kv=-1), "max_kv", 1), (dict(kv_len=None), "kv_len", 1),
                           (dict(kv_len=place(4) + 1), "kv_len", 4), (dict(pages=None), "pages", 1),
                           (dict(pages=place(5) + 2), "pages", 4), (dict(max_pages=-1), "max_pages", 1)):
        refused(lib, size(cache(), batch(**kw)), text, code)
    refused(lib, size(cache(), h=6), "q_heads", 1)
    refused(lib, size(cache(), h=0), "q_heads", 1)
    refused(lib, size(cache(), io=2), "dtype", 3)
    refused(lib, size(cache(), window=-1), "window", 1)
    refused(lib, size(cache(), causal=0, window=5), "window", 5)
    refused(lib, size(cache(), batch(tokens=1 << 29, max_q=1, cu_q=place(12))), "2^31", 5)


def test_append_refusals(lib):
    def call(c=None, b=None, k=None, v=None, q=None, qo=None, qh=8, io=1, rot=None):
        return lib.m3_kv_append(c or cache(), b or batch(), k or rows(7), v or rows(8), q, qo, qh, io, rot, None)
    refused(lib, lib.m3_kv_append(cache(), batch(), None, rows(8), None, None, 0, 1, None, None), "k is NULL", 1)
    refused(lib, call(v=rows(8, p=None)), "v is NULL", 1)
    refused(lib, call(io=9), "dtype", 3)
    refused(lib, call(q=rows(9, 8)), "together", 1)
    refused(lib, call(qo=rows(9, 8)), "together", 1)
    refused(lib, call(q=rows(9, 8), qo=rows(10, 8), qh=0), "q_heads", 1)
    refused(lib, call(q=rows(9, 8), qo=rows(10, 8, head_stride=0)), "q_out", 1)
    refused(lib, call(q=rows(9, 8), qo=rows(9, 8, p=place(9) + 2)), "q_out overlaps q", 1)
    refused(lib, call(q=rows(9, 8), qo=rows(7, 8)), "q_out overlaps k", 1)
    refused(lib, call(q=rows(9, 8), qo=rows(8, 8)), "q_out overlaps v", 1)
    refused(lib, call(q=rows(9, 8), qo=rows(4, 8)), "q_out overlaps kv_len", 1)
    refused(lib, call(rot=rotary(rot=256)), "rot", 1)
    refused(lib, call(k=rows(0)), "cache k overlaps k", 1)
    refused(lib, call(c=cache(v=place(0) + 4096)), "cache k overlaps cache v", 1)
    refused(lib, call(c=cache(k_scale=place(5))), "cache k_scale overlaps pages", 1)
    refused(lib, call(b=batch(batch=1 << 30, tokens=1 << 30, max_q=1 << 20, cu_q=place(12), pages=None, max_pages=0)), "2^31", 5)
    assert call(b=batch(batch=0, tokens=0)) == 0


def test_read_refusals(lib):
    def call(c=None, b=3, first=place(7), count=place(8), pages=place(5), mp=8, mc=10, k=place(9), v=place(10), io=1):
        return lib.m3_kv_read(c or cache(), b, first, count, pages, mp, mc, k, v, io, None)
    refused(lib, call(b=-1), "batch", 1)
    refused(lib, call(mc=-1), "max_count", 1)
    refused(lib, call(io=4), "dtype", 3)
    refused(lib, call(first=None), "first", 1)
    refused(lib, call(count=place(8) + 1), "count", 4)
    refused(lib, call(k=None), "k_out", 1)
    refused(lib, call(v=place(10) + 8), "v_out", 4)
    refused(lib, call(k=place(0)), "k_out overlaps cache k", 1)
    refused(lib, call(v=place(9)), "k_out overlaps v_out", 1)
    refused(lib, call(pages=None), "pages", 1)
    refused(lib, call(b=1 << 20, mc=1 << 20), "2^31", 5)
    assert call(b=0, first=None) == 0 and call(mc=0, k=None) == 0


def test_attend_refusals(lib):
    def call(q=None, out=place(11), lse=None, scale=1.0, ws=None, n=0, b=None, h=8):
        return lib.m3_kv_attend(cache(), b or batch(max_kv=64), q or rows(10, 8), out, lse, h, 1, scale, 1, 0, ws, n, None)
    refused(lib, call(q=rows(10, 8, p=None)), "q is NULL", 1)
    refused(lib, call(out=None), "out is NULL", 1)
    refused(lib, call(out=place(11) + 8), "out", 4)
    refused(lib, call(lse=place(12) + 2), "lse", 4)
    refused(lib, call(scale=float("inf")), "scale", 1)
    refused(lib, call(out=place(10)), "out overlaps q", 1)
    refused(lib, call(lse=place(11)), "out overlaps lse", 1)
    refused(lib, call(out=place(1)), "out overlaps cache v", 1)
    refused(lib, call(lse=place(4)), "lse overlaps kv_len", 1)
    long = batch(max_kv=1 << 17, max_pages=1 << 11)
    need = lib.m3_kv_attend_workspace_size(cache(), long, 8, 1, 1, 0)
    assert need > 0
    refused(lib, call(b=long), "workspace", 7)
    refused(lib, call(b=long, ws=place(13), n=need - 1), "workspace", 7)
    refused(lib, call(b=long, ws=place(13) + 8, n=need), "workspace", 4)
    refused(lib, call(b=long, ws=place(11), n=need), "out overlaps workspace", 1)
    assert call(b=batch(batch=0, tokens=0)) == 0


@pytest.mark.parametrize("b,h,kv,max_q,max_kv", [(1, 16, 4, 1, 131072), (128, 16, 4, 1, 4096), (3, 8, 8, 7, 1000),
                                                 (1, 4, 1, 512, 32768), (4, 32, 8, 2048, 2048), (1000, 8, 8, 1, 64)])
def test_workspace_size(lib, b, h, kv, max_q, max_kv):
    """Bounded by the parts that 512 workgroups can leave (two row tiles of at most 256 rows each) or by 64 parts of
    every row, and a few words a sequence; nothing for shapes that are refused."""
    c = cache(heads=kv, num_pages=1 << 20)
    bt = batch(batch=b, tokens=b * max_q, max_q=max_q, max_kv=max_kv, cu_q=place(12), max_pages=-(-max_kv // 64))
    n = lib.m3_kv_attend_workspace_size(c, bt, h, 1, 1, 0)
    part = 128 * 4 + 8
    assert n <= max(1024 * 32, 64 * h * b * max_q) * part + 16 * (b * max_q * h + 64)
    assert (n > 0) == (b == 1 and max_kv > 30000) or b != 1     # a few rows over a long context are split
    assert lib.m3_kv_attend_workspace_size(c, bt, h + 1 if kv > 1 else 0, 1, 1, 0) == 0


def test_python_refuses_cpu_tensors():
    import torch
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        at.rope(x, torch.zeros(2, dtype=torch.int32), torch.ones(32))
    with pytest.raises(ValueError):
        at.KVCache(x, x, x, x)
    with pytest.raises(ValueError):
        at.KVCache.empty(4, 24, 2, 64, device="cpu")
