"""rope as a step of autograd: gradients of its input against the 64-bit map's, by autograd and by differences."""
import pytest
import torch

from mamba_ssm_scan_amd import attention
from tests import attn_ref as ref
from tests.test_gpu_attention import BF, DEV, F32, gen, normal, turn_bound, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (33, 3, 80, 32), (7, 2, 20, 6), (0, 2, 64, 64)])
def test_gradient(T, H, D, rot, inter, dt):
    g = gen(T + D)
    ms = 1.25
    x = normal(g, T, H, D, dtype=dt).to(DEV).requires_grad_()
    dy = normal(g, T, H, D, dtype=dt)
    pos = torch.randint(0, 4000, (T,), generator=g, dtype=torch.int32)
    f, _ = attention.rope_frequencies(rot, device="cpu")
    y = attention.rope(x, pos.to(DEV), f.to(DEV), interleaved=inter, mscale=ms)
    assert y.requires_grad
    xc = x.detach().cpu()
    want = ref.turn(xc, pos, f, inter, ms)
    within(y, want, turn_bound(xc, want, ms, dt), "y")
    y.backward(dy.to(DEV))
    z = x.detach().cpu().double().requires_grad_()
    (want,) = torch.autograd.grad(ref.turn(z, pos, f, inter, ms), z, dy.double())
    within(x.grad, want, turn_bound(dy, want, ms, dt), "dx")


def test_gradients_reach_weights_and_broadcast_rows():
    """Through a product before it and a sum after it (whose gradient has no strides), on another stream too; the
    gradient's own gradient (the map is linear); and by differences."""
    g = gen(1)
    T, H, D = 12, 2, 32
    f = attention.rope_frequencies(D)[0]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    u, w = normal(g, T, 48).to(DEV), normal(g, 48, H * D).to(DEV).requires_grad_()
    turned = lambda m, **kw: attention.rope((u @ m).view(T, H, D), pos, f, **kw)  # noqa: E731
    turned(w).sum().backward()
    back = ref.turn(torch.ones(T, H, D), pos.cpu(), f.cpu(), backward=True)
    want = u.cpu().double().T @ back.reshape(T, H * D)
    # each entry: T products, each factor off by 2^-22 of at most 2 |u|
    assert (w.grad.cpu().double() - want).abs().max() <= T * 2.0 ** -20 * 2 * u.abs().max().item()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first, w.grad = w.grad, None
    with torch.cuda.stream(side):
        turned(w, stream=side).sum().backward()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(w.grad, first)
    d = normal(g, 48, H * D).to(DEV)
    with torch.no_grad():
        diff = (turned(w + d).double().sum() - turned(w - d).double().sum()) / 2
    assert abs(float(diff - (first.double() * d.double()).sum())) <= 2.0 ** -21 * T * H * D * 48
    x = normal(g, T, H, D).to(DEV).requires_grad_()
    v = normal(g, T, H, D).to(DEV).requires_grad_()
    (dx,) = torch.autograd.grad(attention.rope(x, pos, f), x, v, create_graph=True)
    (dv,) = torch.autograd.grad(dx, v, x.detach())
    assert torch.equal(dv, attention.rope(x.detach(), pos, f))


def test_outside_autograd():
    x = normal(gen(2), 3, 1, 16).to(DEV).requires_grad_()
    f = attention.rope_frequencies(16)[0]
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    with torch.no_grad():
        a = attention.rope(x, pos, f)
    b = attention.rope(x, pos, f, out=torch.empty(3, 1, 16, device=DEV))
    c = attention.rope(x, pos, f)
    assert not a.requires_grad and not b.requires_grad and torch.equal(a, b) and torch.equal(a, c)
