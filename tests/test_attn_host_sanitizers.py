"""The attention layer's host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): the C entry points
of the whole library, device launchers stubbed out, with the attention ABI tests run against that build."""
import os
import subprocess
import sys

import pytest

from tests.test_host_sanitizers import HERE, ROOT, _have_toolchain, host_check


@pytest.mark.skipif(not _have_toolchain(), reason="HIP host headers and runtime library not installed")
def test_attention_abi_under_asan_ubsan(tmp_path):
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
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_attn_abi.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
