"""The attention layer's entry points at the ends of their arguments' ranges, without a GPU; and the same under
AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import subprocess
import sys

import pytest

from mamba_ssm_scan_amd import attention as at
from tests.test_attn_abi import batch, cache, lib, place  # noqa: F401  (lib: the fixture)
from tests.test_host_sanitizers import HERE, ROOT, _have_toolchain, host_check


def need(lib, b, heads, io=1, causal=1, window=0, kv=4, dim=128):
    return lib.m3_kv_attend_workspace_size(cache(heads=kv, headdim=dim, num_pages=1 << 20), b, heads, io, causal, window)


@pytest.mark.parametrize("max_q,tokens", [(1, 3), (7, 21), (300, 900)])
def test_a_window_of_any_size(lib, max_q, tokens):
    """A window longer than every sequence is planned as none is, up to the largest number."""
    b = batch(tokens=tokens, max_q=max_q, max_kv=1 << 17, max_pages=1 << 11, cu_q=place(12))
    want = need(lib, b, 8)
    assert want > 0
    for window in (1 << 17, (1 << 31) - 1, 1 << 31, (1 << 62) + 5, (1 << 63) - 64, (1 << 63) - 1):
        assert need(lib, b, 8, window=window) == want, window
    assert 0 < need(lib, b, 8, window=1 << 14) <= want


@pytest.mark.parametrize("b,h,kv,max_q,max_kv,split", [
    (1, 16, 4, 1, 131072, True),       # a few rows over a long context: even shares
    (128, 16, 4, 1, 4096, False),      # 512 (sequence, head) pairs fill the chip by themselves
    (3, 8, 8, 7, 1000, False),         # 16 tiles of keys: short
    (3, 8, 8, 7, 1100, True),          # 18
    (1, 4, 1, 512, 32768, True),       # a piece of a prompt in 8 workgroups: its keys are split
    (4, 32, 8, 2048, 2048, False),     # prompts that fill the chip
    (1000, 8, 8, 1, 64, False)])
def test_workspace_where_keys_are_split_and_only_there(lib, b, h, kv, max_q, max_kv, split):
    bt = batch(batch=b, tokens=b * max_q, max_q=max_q, max_kv=max_kv, cu_q=place(12), max_pages=-(-max_kv // 64))
    n = need(lib, bt, h, kv=kv)
    assert (n > 0) == split
    # parts: headdim sums and two numbers each, at least two of the rows that a workgroup takes
    assert not split or n >= 2 * 16 * (128 * 4 + 8)


def brute(pa, ta, ha, na, pb, tb, hb, nb, tokens, dim):
    """Whether two sets of rows (bytes; strides in entries of 2 bytes) share a byte, entry by entry."""
    seen = {pa + 2 * (t * ta + h * ha + d) for t in range(tokens) for h in range(na) for d in range(dim)}
    return any(pb + 2 * (t * tb + h * hb + d) in seen for t in range(tokens) for h in range(nb) for d in range(dim))


def test_overlaps_are_found_to_the_entry(lib):
    """Rows of one buffer, interleaved by token and by head in every order: what shares an entry is refused. What
    shares none is accepted by the overlap check; the call then ends at its next check (positions on the output)."""
    import random
    rng = random.Random(7)
    told = {False: 0, True: 0}
    for _ in range(4000):
        tokens, heads, dim = rng.randint(1, 5), rng.randint(1, 4), rng.choice([2, 4, 6])
        parts = rng.randint(2, 4)
        if rng.random() < 0.5:   # [token][head][part][dim] with gaps
            hs = parts * dim + rng.randint(0, 3)
            ts = hs * heads + rng.randint(0, 5)
        else:                    # [head][token][part][dim]
            ts = parts * dim + rng.randint(0, 3)
            hs = ts * tokens + rng.randint(0, 5)
        shift = 2 * rng.randint(-3 * dim - ts, 3 * dim + ts)
        base = place(7)
        x, y = at.M3Rows(base + shift, ts, hs), at.M3Rows(base, ts, hs)
        if shift == 0:
            continue             # in place, which is allowed
        rot = at.M3Rotary(place(6), 2, 0, 1.0)
        s = lib.m3_rope(x, y, tokens, heads, dim, 1, base, rot, 0, None)
        text = lib.m3_last_error().decode()
        assert s == 1 and ("y overlaps x" in text or "y overlaps positions" in text), text
        want = brute(base + shift, ts, hs, heads, base, ts, hs, heads, tokens, dim)
        assert ("y overlaps x" in text) == want, (tokens, heads, dim, ts, hs, shift)
        told[want] += 1
    assert min(told.values()) > 300, told


def test_overlaps_of_parts_of_different_head_counts(lib):
    """q_out against k and v with other head counts: refused where an entry is shared; a call without an overlap ends
    at the next check (q_out on kv_len)."""
    import random
    rng = random.Random(8)
    told = {False: 0, True: 0}
    for _ in range(3000):
        tokens, g, q, dim = rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 6), 16
        hs = rng.choice([1, 2, 3]) * dim + 2 * rng.randint(0, 2)
        ts = hs * (q + 2 * g) + 2 * rng.randint(0, 3)
        base = place(7)
        off = 2 * rng.randint(-ts, ts + hs * g)
        qr = at.M3Rows(base, ts, hs)
        c = cache(heads=g, headdim=dim)
        s = lib.m3_kv_append(c, batch(tokens=tokens, batch=tokens, kv_len=base), at.M3Rows(base + off, ts, hs),
                             at.M3Rows(place(20), ts, hs), qr, qr, q, 1, None, None)
        text = lib.m3_last_error().decode()
        assert s == 1 and ("q_out overlaps k" in text), text
        want = brute(base, ts, hs, q, base + off, ts, hs, g, tokens, dim)
        assert (text == "q_out overlaps k") == want, (tokens, g, q, ts, hs, off, text)
        told[want] += 1
    assert min(told.values()) > 300, told


def _toolchain():
    return _have_toolchain() and not os.environ.get("M3_LIBRARY")


@pytest.mark.skipif(not _toolchain(), reason="HIP host headers and runtime library not installed, or inside that run")
def test_these_under_asan_ubsan(tmp_path):
    out = str(tmp_path / "libm3_attn_hostcheck.so")
    srcs = [os.path.join(host_check.CSRC, f) for f in ("m3_host.cpp", "m3_mixer.cpp", "m3_paths.cpp", "m3_attn_host.cpp")]
    srcs += [os.path.join(HERE, "host_check", f) for f in ("m3_stub_launch.cpp", "m3_attn_stub_launch.cpp")]
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", *host_check.SAN, "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", host_check.CSRC, "-o", out, *srcs,
                    "-L/opt/rocm/lib", "-lamdhip64", "-lhipblaslt", "-Wl,-rpath,/opt/rocm/lib"],
                   check=True, capture_output=True, text=True)
    env = dict(os.environ, LD_PRELOAD=host_check.preload(), M3_LIBRARY=out,
               ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:detect_odr_violation=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_attn_abi_bounds.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
