"""Windows longer than anything held, up to the largest number: as without a window, also where rows lie before the
first position (more rows than tokens held)."""
import pytest
import torch

from tests.test_gpu_attention import BF, DEV, F32, I8, Bench, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,n", [([9, 40], [30, 5]), ([150, 300], [200, 70]), ([2000, 3], [9, 9])], ids=str)
def test_windows_that_reach_past_everything(lens, n, io):
    bench = Bench(2, 1, 64, 16, max(lens), I8, seed=sum(n))
    bench.append(list(lens))
    q = normal(bench.g, sum(n), 2, 64, dtype=io).to(DEV)
    cu = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=DEV)
    kw = dict(cu_q=cu, max_q=max(n), lse=True)
    want = bench.cache.attend(q, bench.kv_len(), bench.pages, **kw)
    for window in (max(lens), 1 << 20, (1 << 31) - 1, 1 << 31, 1 << 40, (1 << 63) - 64, (1 << 63) - 1):
        for got, w in zip(bench.cache.attend(q, bench.kv_len(), bench.pages, window=window, **kw), want):
            assert torch.equal(got, w), window
