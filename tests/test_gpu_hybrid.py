"""The hybrid stack (examples/hybrid_stack.py): mixers and attention over the 8-bit cache, prompt and steps together."""
import importlib.util
import os

import pytest
import torch

from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("hybrid_stack", os.path.join(ROOT, "examples", "hybrid_stack.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_steps_continue_a_prompt(fmt):
    """A prompt of 96 and 5 steps give what a prompt of 101 gives at those tokens, to the bar of the mixers' bf16
    contracts (2e-2 of the largest entry) for each of the stack's layers, whose errors add (6 layers, two of the bars
    for the cache: a block's codes are rounded again when its scale grows)."""
    ex = _example()
    u = torch.randn((2, 101, 256), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").bfloat16()
    kw = dict(groups=1, mixers=5, d_model=256, mixer_heads=4, heads=4, kv_heads=2, page_size=16, room=112,
              fmt=ex.FORMATS[fmt])
    whole = ex.HybridStack(2, **kw).prompt(u)
    stack = ex.HybridStack(2, **kw)
    head = stack.prompt(u[:, :96].contiguous())
    assert (head.float() - whole[:, :96].float()).abs().max() <= 8 * 2e-2 * whole.float().abs().max()
    for k in range(5):
        x = stack.step(u[:, 96 + k].contiguous())
        err = (x.float() - whole[:, 96 + k].float()).abs().max() / whole[:, 96 + k].float().abs().max()
        print(f"  step {k}: {float(err):.2e}", flush=True)
        assert err <= 8 * 2e-2


def test_attention_layer_against_64_bits():
    """One attention layer of the stack, its projections included, from bf16 weights and tokens."""
    ex = _example()
    layer = ex.AttentionLayer(128, 4, 2, 64, 16, 16, torch.int8, seed=3)
    u = torch.randn((40, 128), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").bfloat16()
    pages = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    kv_len = torch.tensor([25, 15], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 25, 40], dtype=torch.int32, device="cuda")
    got = layer(u, kv_len, pages, cu_q=cu, max_q=25).cpu().double()
    uc, f = u.cpu().double(), layer.inv_freq.cpu()
    qkv = (uc @ layer.w_qkv.cpu().double().T).view(40, 8, 64)
    at = 0
    for n in (25, 15):
        pos = torch.arange(n)
        rows = qkv[at:at + n]
        q, k = ref.turn(rows[:, :4], pos, f), ref.turn(rows[:, 4:6], pos, f)
        o, _, _, _ = ref.attend(q, pos, k, rows[:, 6:], 64 ** -0.5)
        want = o.reshape(n, 256) @ layer.w_out.cpu().double().T
        # int8 blocks: half a step of amax / 127 an entry, about 1 % of a value's size; bf16 in between
        assert (got[at:at + n] - want).abs().max() <= 3e-2 * want.abs().max()
        at += n
