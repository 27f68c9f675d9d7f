"""The joint's host code under AddressSanitizer and UndefinedBehaviorSanitizer, and its kernels' LDS and scratch from the
metadata of the built code (CPU only)."""
import os
import subprocess
import sys

import pytest

from tests.test_host_sanitizers import HERE, ROOT, _have_toolchain, host_check
from tests.test_kernel_resources import LDS_PER_CU, _code_objects, _kernels


@pytest.mark.skipif(not _have_toolchain(), reason="HIP host headers and runtime library not installed")
def test_norm_abi_under_asan_ubsan(tmp_path):
    out = str(tmp_path / "libm3_norm_hostcheck.so")
    srcs = [os.path.join(host_check.CSRC, f) for f in ("m3_host.cpp", "m3_mixer.cpp", "m3_paths.cpp", "m3_norm_host.cpp")]
    srcs += [os.path.join(HERE, "host_check", f) for f in ("m3_stub_launch.cpp", "m3_norm_stub_launch.cpp")]
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", *host_check.SAN, "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", host_check.CSRC, "-o", out, *srcs,
                    "-L/opt/rocm/lib", "-lamdhip64", "-lhipblaslt", "-Wl,-rpath,/opt/rocm/lib"],
                   check=True, capture_output=True, text=True)
    env = dict(os.environ, LD_PRELOAD=host_check.preload(), M3_LIBRARY=out,
               ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:detect_odr_violation=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_norm_abi.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail


def test_kernel_resources(tmp_path):
    rows = [k for obj in _code_objects() if os.path.basename(obj) == "m3_norm.o" for k in _kernels(obj, str(tmp_path))]
    for n in ("joint_kernel", "joint_back_kernel", "joint_sums_kernel"):
        assert any(n in k for k, _, _ in rows), n
    for name, lds, scratch in rows:
        assert lds <= LDS_PER_CU and scratch == 0, (name, lds, scratch)
