"""A hybrid stack served end to end: groups of mixer blocks with one attention layer each.

The pages' 5:1 hybrid ("Mamba-3架构技术解析：新一代语言建模的范式转移", §4.2): five mixer blocks (binding.Mixer), then one
attention layer over the paged 8-bit cache (attention.KVCache), every layer behind an RMS norm and a residual. Random
weights: what it shows is the calls and how their states go together.

    python examples/hybrid_stack.py [--batch 4] [--prompt 512] [--steps 32] [--format int8|fp8]

One page table and one vector of lengths serve every attention layer: the lengths are raised once a step, on the
device, before the layers run.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mamba_ssm_scan_amd import attention, binding, inputs  # noqa: E402

FORMATS = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}


def rms_norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class AttentionLayer:
    """One fused projection to q, k, v; the rotation and the cache's append in one launch; attention; the projection
    back. The heads of q, k and v are used where the projection left them."""

    def __init__(self, d_model, heads, kv_heads, head_dim, num_pages, page_size, fmt, seed, window=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = (heads + 2 * kv_heads) * head_dim
        self.w_qkv = (torch.randn((rows, d_model), generator=g, device="cuda") * d_model ** -0.5).to(torch.bfloat16)
        self.w_out = (torch.randn((d_model, heads * head_dim), generator=g, device="cuda")
                      * (heads * head_dim) ** -0.5).to(torch.bfloat16)
        self.cache = attention.KVCache.empty(num_pages, page_size, kv_heads, head_dim, dtype=fmt)
        self.inv_freq, self.mscale = attention.rope_frequencies(head_dim)
        self.heads, self.kv_heads, self.head_dim, self.window = heads, kv_heads, head_dim, window

    def __call__(self, u, kv_len, pages, cu_q=None, max_q=1):
        """u [tokens][d_model]: the rows of the batch's new tokens, sequence after sequence."""
        H, G, D = self.heads, self.kv_heads, self.head_dim
        qkv = (u @ self.w_qkv.T).view(-1, H + 2 * G, D)
        q = self.cache.append(qkv[:, H:H + G], qkv[:, H + G:], kv_len, pages, cu_q=cu_q, max_q=max_q, q=qkv[:, :H],
                              inv_freq=self.inv_freq, mscale=self.mscale)
        o = self.cache.attend(q, kv_len, pages, cu_q=cu_q, max_q=max_q, window=self.window)
        return o.view(u.shape[0], H * D) @ self.w_out.T


class HybridStack:
    """`groups` times (`mixers` mixer blocks, one attention layer), for a batch of sequences of one prompt length."""

    def __init__(self, batch, groups=1, mixers=5, d_model=512, mixer_heads=8, heads=8, kv_heads=2, head_dim=64,
                 page_size=64, room=4096, fmt=torch.int8, seed=0):
        self.batch, self.d_model = batch, d_model
        per = -(-room // page_size)
        # every sequence gets its own pages; a server would hand them out as the sequences grow
        self.pages = torch.randperm(batch * per, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.pages = self.pages.view(batch, per).cuda()
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.layers = []
        for g in range(groups):
            for m in range(mixers):
                w = inputs.mixer_inputs(batch=1, seqlen=1, d_model=d_model, heads=mixer_heads, groups=1, headdim=64,
                                        dstate=128, rank=1, wid=9000 + 100 * g + m + seed, device="cuda")
                mixer = binding.Mixer(w)
                self.layers.append((mixer, mixer.decode_state(batch)))
            self.layers.append((AttentionLayer(d_model, heads, kv_heads, head_dim, batch * per, page_size, fmt,
                                               seed=1000 + g + seed), None))

    def prompt(self, u):
        """u [batch][tokens][d_model] -> the stack's output, states and caches filled."""
        b, L, dm = u.shape
        self.kv_len.fill_(L)
        cu = torch.arange(0, (b + 1) * L, L, dtype=torch.int32, device="cuda")
        x = u
        for layer, state in self.layers:
            y = rms_norm(x)
            if state is not None:
                y, _ = layer.prefill(y, state=state)
            else:
                y = layer(y.reshape(b * L, dm), self.kv_len, self.pages, cu_q=cu, max_q=L).view(b, L, dm)
            x = x + y
        return x

    def step(self, u):
        """u [batch][d_model]: one token a sequence."""
        self.kv_len.add_(1)
        x = u
        for layer, state in self.layers:
            y = rms_norm(x)
            x = x + (layer.decode_step(state, y) if state is not None else layer(y, self.kv_len, self.pages))
        return x


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--groups", type=int, default=2)
    ap.add_argument("--format", choices=sorted(FORMATS), default="int8")
    a = ap.parse_args()
    stack = HybridStack(a.batch, groups=a.groups, room=a.prompt + a.steps, fmt=FORMATS[a.format])
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.randn((a.batch, a.prompt + a.steps, stack.d_model), generator=g, device="cuda").to(torch.bfloat16)
    for what in ("first", "again"):   # the first pass also chooses the mixers' matrix products
        torch.cuda.synchronize()
        t = time.perf_counter()
        stack.prompt(u[:, :a.prompt].contiguous())
        torch.cuda.synchronize()
        t1 = time.perf_counter()
        for k in range(a.steps):
            x = stack.step(u[:, a.prompt + k].contiguous())
        torch.cuda.synchronize()
        t2 = time.perf_counter()
        print(f"{what}: prompt {a.batch} x {a.prompt} in {1e3 * (t1 - t):.2f} ms, {a.steps} steps at "
              f"{1e6 * (t2 - t1) / a.steps:.0f} us; last output {tuple(x.shape)}, rms {float(x.float().square().mean().sqrt()):.3f}",
              flush=True)


if __name__ == "__main__":
    main()
