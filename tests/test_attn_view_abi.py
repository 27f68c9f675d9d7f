"""Checks of the attention view's C entry points that need no GPU (pointers are fake, never dereferenced)."""
import ctypes  # noqa: F401
import os
import subprocess
import sys

import pytest

from mamba_ssm_scan_amd import attention as at
from tests.test_attn_abi import batch, cache, lib, place, refused, rows  # noqa: F401
from tests.test_host_sanitizers import HERE, ROOT, _have_toolchain, host_check


def view(**kw):
    d = dict(causal=1, window=0, sinks=0, groups=2, max_prefix=4, group_start=place(14), prefix_count=place(15),
             prefix_pages=place(16))
    d.update(kw)
    return at.M3KvView(*[d[n] for n, _ in at.M3KvView._fields_])


def call(lib, v, b=None, out=place(11), lse=None, ws=None, n=0, h=8, c=None):  # noqa: F811
    return lib.m3_kv_attend_view(c or cache(), b or batch(max_kv=64), v, rows(10, 8), out, lse, h, 1, 1.0, ws, n, None)


def test_refusals(lib):  # noqa: F811
    refused(lib, call(lib, None), "view is NULL", 1)
    for kw, text, code in ((dict(window=-1), "window", 1), (dict(causal=0, window=5), "window", 5), (dict(sinks=-1), "sinks", 1),
                           (dict(groups=-1), "groups", 1), (dict(groups=(1 << 30) + 1), "groups", 1),
                           (dict(max_prefix=-1), "max_prefix", 1), (dict(max_prefix=(1 << 31) + 1), "max_prefix", 1),
                           (dict(group_start=None), "group_start is NULL", 1), (dict(prefix_count=None), "prefix_count", 1),
                           (dict(prefix_pages=None), "prefix_pages", 1), (dict(group_start=place(14) + 2), "not 4-byte", 4),
                           (dict(prefix_count=place(15) + 1), "not 4-byte", 4), (dict(prefix_pages=place(16) + 2), "not 4-byte", 4)):
        refused(lib, call(lib, view(**kw)), text, code)
    refused(lib, call(lib, view(), out=place(16)), "out overlaps prefix_pages", 1)
    refused(lib, call(lib, view(), lse=place(15)), "lse overlaps prefix_count", 1)
    refused(lib, call(lib, view(), out=place(14)), "out overlaps group_start", 1)
    for v in (view(), view(groups=1, group_start=None), view(groups=0, group_start=None, prefix_count=None, prefix_pages=None),
              view(max_prefix=0, prefix_pages=None), view(window=1 << 62, sinks=1 << 62), view(max_prefix=1 << 31)):
        assert call(lib, v, b=batch(batch=0, tokens=0)) == 0


def test_workspace(lib):  # noqa: F811
    size = lib.m3_kv_attend_view_workspace_size
    assert size(cache(), batch(), view(sinks=-1), 8, 1) == 0
    plain = dict(groups=0, group_start=None, prefix_count=None, prefix_pages=None, max_prefix=0)
    long = batch(max_kv=1 << 17, max_pages=1 << 11)
    assert size(cache(), long, view(**plain), 8, 1) == lib.m3_kv_attend_workspace_size(cache(), long, 8, 1, 1, 0) > 0
    need = size(cache(), long, view(max_prefix=1 << 10), 8, 1)
    assert need > 0
    refused(lib, call(lib, view(max_prefix=1 << 10), b=long), "workspace", 7)
    refused(lib, call(lib, view(max_prefix=1 << 10), b=long, ws=place(13), n=need - 1), "workspace", 7)
    refused(lib, call(lib, view(max_prefix=1 << 10), b=long, ws=place(16), n=need), "workspace overlaps prefix_pages", 1)


@pytest.mark.skipif(not _have_toolchain() or "M3_LIBRARY" in os.environ, reason="HIP host headers not installed, or run inside")
def test_under_asan_ubsan(tmp_path):
    out = str(tmp_path / "libm3_attn_view_hostcheck.so")
    srcs = [os.path.join(host_check.CSRC, f) for f in ("m3_host.cpp", "m3_mixer.cpp", "m3_paths.cpp", "m3_attn_host.cpp")]
    srcs += [os.path.join(HERE, "host_check", f) for f in ("m3_stub_launch.cpp", "m3_attn_stub_launch.cpp")]
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", *host_check.SAN, "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", host_check.CSRC, "-o", out, *srcs,
                    "-L/opt/rocm/lib", "-lamdhip64", "-lhipblaslt", "-Wl,-rpath,/opt/rocm/lib"],
                   check=True, capture_output=True, text=True)
    env = dict(os.environ, LD_PRELOAD=host_check.preload(), M3_LIBRARY=out,
               ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:detect_odr_violation=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_attn_view_abi.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
