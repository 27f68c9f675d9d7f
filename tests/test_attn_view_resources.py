"""LDS and scratch of the attention kernels' instances for sinks and prefixes, from the metadata of the built code (CPU
only)."""
import os

from tests.test_attn_kernel_resources import dynamic_lds
from tests.test_kernel_resources import LDS_PER_CU, _code_objects, _kernels

KERNELS = {"m3_kv_attend_view": "attend_rows_kernel", "m3_kv_attend_parts": "attend_merge_kernel",
           "m3_kv_attend_tile_view": "attend_tile_kernel"}


def test_view_kernels(tmp_path):
    for obj in _code_objects():
        base = os.path.splitext(os.path.basename(obj))[0]
        if base not in KERNELS:
            continue
        rows = _kernels(obj, str(tmp_path))
        assert any(KERNELS[base] in n for n, _, _ in rows), base
        for name, lds, scratch in rows:
            assert lds + dynamic_lds(name) <= LDS_PER_CU and scratch == 0, (name, lds, dynamic_lds(name), scratch)
