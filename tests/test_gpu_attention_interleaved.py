"""q, k and v interleaved by head in one projection, [token][head][q, k, v][dim]: used where they lie, q in place."""
import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests.test_gpu_attention import BF, DEV, F32, I8, Bench, gen, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 21])
def test_parts_interleaved_by_head(T, io):
    H, D = 3, 64
    f = attention.rope_frequencies(D)[0]
    x = normal(gen(T), T, H, 3, D, dtype=io).to(DEV)
    q, k, v = x.unbind(2)
    bench = Bench(1, H, D, 16, 32, I8)
    other = attention.KVCache.empty(bench.n_pages, 16, H, D)
    kv, cu = torch.tensor([T], dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV)
    kw = dict(cu_q=cu, max_q=T, inv_freq=f)
    before = x.clone()
    want = bench.cache.append(k.contiguous(), v.contiguous(), kv, bench.pages, q=q.contiguous(), **kw)
    got = other.append(k, v, kv, bench.pages, q=q, q_out=q, **kw)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
    assert torch.equal(x[:, :, 1:], before[:, :, 1:])
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    for a, b in zip(bench.cache.read(zero, kv, bench.pages, T), other.read(zero, kv, bench.pages, T)):
        assert torch.equal(a, b)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    y = attention.rope(x[:, :, 1], pos, f, out=x[:, :, 2])       # from one part into another
    assert torch.equal(y, attention.rope(before[:, :, 1].contiguous(), pos, f))
