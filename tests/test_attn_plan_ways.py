"""Which way attend's plan takes the calls of the GPU tests of shared prefixes, from the host code alone: those tests look
for the kernels that a call launched, which says nothing where the profiler sees none."""
import ctypes
import os
import subprocess

import pytest
import torch

from mamba_ssm_scan_amd import attention as at
from tests import test_gpu_attention_parts as parts
from tests.test_attn_abi import batch, cache, place, rows
from tests.test_gpu_attention import BF, F32
from tests.test_host_sanitizers import HERE, ROOT, _have_toolchain, host_check

pytestmark = pytest.mark.skipif(not _have_toolchain(), reason="HIP host headers and runtime library not installed")

PARTS, PREFIX_TILE, ITEMS = 1, 2, 4
WAYS = {"items": PARTS | ITEMS, "join": PARTS | PREFIX_TILE, "merge": PARTS | PREFIX_TILE | ITEMS}


@pytest.fixture(scope="module")
def noting(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan") / "libm3_attn_plan.so")
    srcs = [os.path.join(host_check.CSRC, f) for f in ("m3_host.cpp", "m3_mixer.cpp", "m3_paths.cpp", "m3_attn_host.cpp")]
    srcs += [os.path.join(HERE, "host_check", f) for f in ("m3_stub_launch.cpp", "m3_attn_plan_launch.cpp")]
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"), "-I", host_check.CSRC, "-o", out, *srcs,
                    "-L/opt/rocm/lib", "-lamdhip64", "-lhipblaslt", "-Wl,-rpath,/opt/rocm/lib"],
                   check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(out)
    real = at._lib()
    for name in ("m3_kv_attend_view", "m3_kv_attend_view_workspace_size"):
        getattr(lib, name).argtypes, getattr(lib, name).restype = getattr(real, name).argtypes, getattr(real, name).restype
    return lib


def way(lib, kv, H, D, page, io, n, tokens, max_q, room, groups, starts):
    """The call of that many sequences and rows; page table and prefix table of `room` tokens."""
    c = cache(heads=kv, headdim=D, page_size=page, num_pages=1 << 16)
    wide = room // page
    b = batch(batch=n, tokens=tokens, max_pages=wide, max_q=max_q, max_kv=room, cu_q=None if tokens == n else place(7))
    v = at.M3KvView(1, 0, 0, groups, wide, place(14) if starts else None, place(15), place(16))
    code = 0 if io == F32 else 1
    size = lib.m3_kv_attend_view_workspace_size(c, b, v, H, code)
    assert lib.m3_kv_attend_view(c, b, v, rows(10, H, D), place(11), None, H, code, D ** -0.5, place(13) if size else None,
                                 size, None) == 0
    return lib.m3_noted_plan()


def the_rows(case):
    """The rows of each sequence as test_ways draws them."""
    _, kv, H, D, page, fmt, io, batch_, rows_, counts, room, tail = case
    g = torch.Generator().manual_seed(batch_ + D + H)
    torch.randint(1, tail, (batch_,), generator=g)
    n = [1] * batch_ if rows_ == 1 else torch.randint(0, rows_ + 1, (batch_,), generator=g).tolist()
    if rows_ > 1:
        n[0], n[5] = rows_, 0
    return n


@pytest.mark.parametrize("case", parts.CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_the_cases_of_each_way(noting, case):
    form, kv, H, D, page, fmt, io, n, rows_, counts, room, tail = case
    r = the_rows(case)
    tokens = sum(r)
    assert tokens != n or rows_ == 1                     # (else cu_q could not be told from none here)
    assert way(noting, kv, H, D, page, io, n, tokens, max(r), room, len(counts), len(counts) > 1) == WAYS[form]


def test_every_way_and_row_count_is_among_them(noting):
    seen = set()
    for case in parts.CASES:
        form, kv, H, D, page, fmt, io, n, rows_, counts, room, tail = case
        r = the_rows(case)
        way(noting, kv, H, D, page, io, n, sum(r), max(r), room, len(counts), len(counts) > 1)
        seen.add((form, noting.m3_noted_prefix_rows(), io == F32))
    assert {f for f, _, _ in seen} == set(parts.FORMS)
    assert {(f, x) for f, _, x in seen} >= {("items", True), ("items", False), ("join", True), ("join", False), ("merge", True)}
    assert {k for f, k, x in seen if f != "items" and not x} >= {64, 128, 256}


@pytest.mark.parametrize("form,n,H,kv", [("items", 16, 8, 2), ("join", 130, 16, 4), ("merge", 60, 64, 8)])
def test_the_sizes_that_the_other_tests_take(noting, form, n, H, kv):
    """Groups and rows of no group, spoiled values, graphs and streams; rows left as they were (fp32)."""
    for groups, starts in ((3, True), (2, True), (1, False)):
        assert way(noting, kv, H, 64, 16, BF, n, n, 1, 8192, groups, starts) == WAYS[form]
    assert way(noting, kv, H, 64, 16, F32, n, n + 20, 2, 8192, 1, False) & PARTS
