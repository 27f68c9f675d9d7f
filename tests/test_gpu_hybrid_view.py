"""The hybrid stack (examples/hybrid_stack.py) through the joint's kernels, under a window with sinks, and behind a prompt
that its sequences share: the calls together, as a user makes them."""
import pytest
import torch

from mamba_ssm_scan_amd import attention, norm
from tests.test_gpu_attention import BF, DEV, gen, normal
from tests.test_gpu_hybrid import _example

pytestmark = pytest.mark.gpu


def tokens(batch, L, d, seed):
    return torch.randn((batch, L, d), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


KW = dict(groups=1, mixers=2, d_model=256, mixer_heads=4, heads=4, kv_heads=2, page_size=16)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_steps_continue_a_prompt_under_a_window_with_sinks(fmt):
    """A prompt of 96 and 5 steps give what a prompt of 101 gives, to the stack's own bar (3 layers at 2e-2 and two for the
    cache, as tests/test_gpu_hybrid.py)."""
    ex = _example()
    u = tokens(2, 101, 256, 5)
    kw = dict(KW, room=112, fmt=ex.FORMATS[fmt], window=24, sinks=3)
    whole = ex.HybridStack(2, **kw).prompt(u)
    stack = ex.HybridStack(2, **kw)
    stack.prompt(u[:, :96].contiguous())
    for k in range(5):
        x = stack.step(u[:, 96 + k].contiguous())
        assert (x.float() - whole[:, 96 + k].float()).abs().max() <= 5 * 2e-2 * whole.float().abs().max()
    plain = ex.HybridStack(2, **dict(kw, window=0)).prompt(u)
    assert not torch.equal(plain, whole)


@pytest.mark.parametrize("batch,L", [(3, 100), (18, 2100)])
def test_a_shared_prompt_is_the_prompt_of_each(batch, L):
    """Steps behind a shared prompt (one pass over its pages, and parts) against the same prompt held by each sequence; the
    prompt's pages are then the first sequence's alone."""
    ex = _example()
    u, steps = tokens(1, L, 256, 6), tokens(batch, 4, 256, 7)
    kw = dict(KW, room=L + 20, fmt=torch.int8)
    own = ex.HybridStack(batch, **kw)
    a = own.prompt(u.expand(batch, L, 256).contiguous())
    stack = ex.HybridStack(batch, **kw)
    b = stack.shared_prompt(u)
    bar = 5 * 2e-2 * a.float().abs().max()
    assert (a[:1].float() - b.float()).abs().max() <= bar
    for k in range(4):
        x, y = own.step(steps[:, k].contiguous()), stack.step(steps[:, k].contiguous())
        assert (x.float() - y.float()).abs().max() <= bar, k


def test_a_training_step_of_an_attention_block():
    """Norm, projection, rotation, plain attention, the joint and the next norm, with gradients into every weight, against
    64 bits."""
    T, H, D = 20, 2, 32
    W = H * D
    g = gen(8)
    leaf = [t.to(DEV).requires_grad_() for t in (normal(g, T, W), normal(g, W, 3 * W) / 8, normal(g, W, W) / 8,
                                                 1 + 0.1 * normal(g, W), 1 + 0.1 * normal(g, W), normal(g, W) / 4)]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    f = attention.rope_frequencies(D)[0]
    up = normal(g, T, W).to(DEV)

    def block(x, w_qkv, w_out, w1, w2, s, joint, rope, p, mask):
        y = joint(x, weight=w1)
        q, k, v = (y @ w_qkv).view(T, 3, H, D).unbind(1)
        q, k = rope(q, p), rope(k, p)
        a = (q.transpose(0, 1) @ k.permute(1, 2, 0).contiguous() * D ** -0.5).masked_fill(mask, -1e30).softmax(-1)
        o = (a @ v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(T, W) @ w_out
        h, y = joint(x, o, gate=x, scale=s, post_weight=w1, weight=w2)
        return (h * y).sum() + (y * p_up(up, h)).sum()

    def p_up(u, like):
        return u.to(like.device, like.dtype)

    def plain(x, o=None, gate=None, scale=None, post_weight=None, weight=None):
        n = lambda t, w: t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w  # noqa: E731
        if o is None:
            return n(x, weight)
        h = x + n(o, post_weight) * gate * torch.sigmoid(gate) * scale
        return h, n(h, weight)

    def turn(x, p):
        th = p.double()[:, None] * f.cpu().double()
        c, s = th.cos()[:, None], th.sin()[:, None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    mask = torch.ones(T, T, dtype=torch.bool).triu(1)
    loss = block(*leaf, norm.residual_norm, lambda t, p: attention.rope(t, p, f), pos, mask.to(DEV))
    got = torch.autograd.grad(loss, leaf)
    copies = [t.detach().cpu().double().requires_grad_() for t in leaf]
    want = torch.autograd.grad(block(*copies, plain, turn, pos.cpu(), mask), copies)
    for a, b in zip(got, want):
        # chains of about a dozen fp32 steps of up to 64 terms: some thousands of roundings of the largest entries
        assert (a.cpu().double() - b).abs().max() <= 4000 * 2.0 ** -24 * b.abs().max()
