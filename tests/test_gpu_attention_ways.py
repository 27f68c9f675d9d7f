"""That the profiler names the kernels of attend's launches here: the tests that tell a call's way by them
(test_gpu_attention_parts.py, test_gpu_attention_poison.py) pass without a word where it does not, and the plan's choice then
rests on test_attn_plan_ways.py alone."""
import pytest

from mamba_ssm_scan_amd import attention
from tests.test_gpu_attention import BF, DEV, I8, normal
from tests.test_gpu_attention_parts import FORMS, bench, launched
from tests.test_gpu_attention_view import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,batch,H,kv", [("items", 16, 8, 2), ("join", 130, 16, 4), ("merge", 60, 64, 8)])
def test_launches_are_named(form, batch, H, kv):
    import torch
    page, D = 16, 64
    b = bench(batch, kv, D, page, I8, [40 * page + 3 + i % 30 for i in range(batch)], seed=9)
    q = normal(b.g, batch, H, D, dtype=BF).to(DEV)
    wide = torch.full((1, 512), -1, dtype=torch.int32, device=DEV)
    wide[0, :40] = b.pages[0, :40]
    pages = torch.full((batch, 512), -1, dtype=torch.int32, device=DEV)
    pages[:, :b.pages.shape[1]] = b.pages
    prefix = attention.SharedPrefix(wide, ints([40]))
    _, names = launched(lambda: b.cache.attend(q, b.kv_len(), pages, prefix=prefix))
    if not names:
        pytest.skip("the profiler sees no launches here")
    assert tuple(names) == FORMS[form]
