"""The attention layer's entry points at the ends of their arguments' ranges, without a GPU; and the same under
AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import subprocess
import sys

import pytest

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
