"""LDS and scratch of every instance of the attention layer's kernels, from the metadata of the built code (CPU only).

Static LDS and the dynamic LDS that each launch asks for fit a compute unit's 160 KiB; no instance has scratch."""
import os
import re

from tests.test_kernel_resources import LDS_PER_CU, _code_objects, _kernels

KERNELS = {"m3_rope": ["rope_wide_kernel", "rope_any_kernel"], "m3_kv_append": ["append_kernel", "read_kernel"],
           "m3_kv_attend": ["attend_rows_kernel", "attend_join_kernel"], "m3_kv_attend_tile": ["attend_tile_kernel"]}


def dynamic_lds(name):
    m = re.search(r"attend_tile_kernelI\w*?ELb[01]ELi(\d+)E", name)
    if m:                       # two images of K and of V, 64 keys of 2-byte entries
        return 4 * 64 * int(m.group(1)) * 2
    if "append_kernel" in name:  # 16 fp32 rows a wave (4 waves up to headdim 128, else 2) and 16 tokens' angles
        return max(4 * 16 * 128 * 4 + 16 * 64 * 8, 2 * 16 * 256 * 4 + 16 * 128 * 8)
    return 0


def test_attention_kernels(tmp_path):
    rows = []
    for obj in _code_objects():
        base = os.path.splitext(os.path.basename(obj))[0]
        if base in KERNELS:
            rows += [(base, *k) for k in _kernels(obj, str(tmp_path))]
    for base, names in KERNELS.items():
        for n in names:
            assert any(b == base and n in k for b, k, _, _ in rows), n
    for base, name, lds, scratch in rows:
        assert lds + dynamic_lds(name) <= LDS_PER_CU, (name, lds, dynamic_lds(name))
        assert scratch == 0, (name, scratch)
    assert any(dynamic_lds(n) == 131072 for _, n, _, _ in rows)
    print(f"{len(rows)} instances")
