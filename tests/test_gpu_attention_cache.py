"""What a KVCache is made of stays: calls go to the memory that its tensors show."""
import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests.test_gpu_attention import DEV, F8, I8, gen, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [I8, F8], ids=["int8", "e4m3"])
def test_tensors_of_a_cache_are_not_replaced(fmt):
    cache = attention.KVCache.empty(2, 16, 1, 32, dtype=fmt)
    for name in ("k", "v", "k_scale", "v_scale"):
        t = getattr(cache, name)
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.empty_like(t))
        assert getattr(cache, name) is t
    x = normal(gen(1), 1, 1, 32).to(DEV)
    one, page = torch.ones(1, dtype=torch.int32, device=DEV), torch.ones(1, 1, dtype=torch.int32, device=DEV)
    cache.append(x, x, one, page)
    again = attention.KVCache(*(getattr(cache, n).clone() for n in ("k", "v", "k_scale", "v_scale")))
    for a, b in zip(cache.read(one - 1, one, page, 1), again.read(one - 1, one, page, 1)):
        assert torch.equal(a, b) and (a - x).abs().max() <= x.abs().max() / (127 if fmt == I8 else 16)
    cache.k.view(I8)[1].zero_()                              # contents may change
    assert not cache.read(one - 1, one, page, 1)[0].any()
