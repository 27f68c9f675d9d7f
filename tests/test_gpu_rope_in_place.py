"""rope in place of rows with a history: values and gradients as into an output of its own."""
import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests.test_gpu_attention import BF, DEV, F32, gen, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", ["rows", "view", "part"])
def test_in_place(form, dt):
    """Rows of their own, a view of a product's result, a part of a fused projection beside others that are used as well."""
    g = gen(3)
    T, H, D = 37, 4, 48
    f, ms = attention.rope_frequencies(D)
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32).to(DEV)
    leaf = normal(g, T, 3 * H * D, dtype=dt).to(DEV).requires_grad_()
    dy = normal(g, T, 3 * H * D, dtype=dt).to(DEV)

    def run(in_place):
        every = leaf * 1.5
        if form == "part":
            x = every.view(T, H, 3, D)[:, :, 1]
        else:
            x = every[:, :H * D].reshape(T, H, D) if form == "rows" else every[:, :H * D].unflatten(1, (H, D))
        y = attention.rope(x, pos, f, mscale=ms, out=x if in_place else None)
        assert (y is x) == in_place
        d = dy[:, :H * D].reshape(T, H, D)
        loss = (y * d).sum()
        if form == "part":
            z = every.view(T, H, 3, D)
            loss = loss + (z[:, :, 0] * dy.view(T, H, 3, D)[:, :, 0]).sum()
        return y.detach().clone(), torch.autograd.grad(loss, leaf)[0]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)
