"""A decoder layer's step around the MoE layer: norm, projections, rotary positions, the 8-bit cache, attention
over it, and the routed experts, first for prompts of two sequences and then token by token.

    python examples/decoder_step.py

The MoE layer has the tiny geometry (hidden 256); the attention around it 4 query heads and 2 kv heads of 64.
The projections are plain matrix products with random weights.  At the end the tokens that were decoded one by
one are run again as a prompt; both ways see the same cache contents but for the blocks' scales, so their
results agree to the cache's 8 bits.
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import int4_routed_expert_gb300 as m  # noqa: E402
from workloads import CONFIGS  # noqa: E402
from workloads.gen import gen_layer  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 4, 2, 64, 16


class DecoderLayer:
    def __init__(self, max_tokens: int, max_kv_len: int, n_seqs: int, device: str = "cuda:0", seed: int = 7):
        wl = CONFIGS["tiny"]
        g = torch.Generator(device)
        g.manual_seed(seed)
        H = wl.shape.hidden
        self.moe = m.MoELayer(gen_layer(wl, device=device), max_tokens)
        self.rope = m.Rope(DIM, theta=1e6, scaling="yarn", factor=4.0, original_len=4096)
        pages_each = -(-max_kv_len // PAGE)
        self.cache = m.KVCache.empty(n_seqs * pages_each, PAGE, KV_HEADS, DIM, n_q_heads=HEADS, max_seqs=n_seqs,
                                     max_tokens=max_tokens, max_kv_len=max_kv_len, device=device)
        # sequence b owns pages b, n_seqs + b, ...
        self.table = (torch.arange(pages_each, device=device, dtype=torch.int32)[None] * n_seqs +
                      torch.arange(n_seqs, device=device, dtype=torch.int32)[:, None]).contiguous()
        self.w_qkv = torch.randn(H, (HEADS + 2 * KV_HEADS) * DIM, device=device, generator=g).bfloat16() * H ** -0.5
        self.w_out = torch.randn(HEADS * DIM, H, device=device, generator=g).bfloat16() * H ** -0.5
        self.gamma = torch.ones(H, device=device)
        self.lens = [0] * n_seqs
        self.device = device

    def step(self, x, news):
        """x [tokens, hidden] fp32: the next news[b] tokens of each sequence; returns the layer's output."""
        n_seqs = len(news)
        self.lens = [a + b for a, b in zip(self.lens, news)]
        i32 = dict(device=self.device, dtype=torch.int32)
        batch = m.SeqBatch(torch.tensor([sum(news[:b]) for b in range(n_seqs + 1)], **i32),
                           torch.tensor(self.lens, **i32), self.table, sum(news), max(news), max(self.lens))
        pos = torch.cat([torch.arange(n - k, n, **i32) for n, k in zip(self.lens, news)])
        normed = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)).bfloat16()
        qkv = (normed @ self.w_qkv).unflatten(1, (HEADS + 2 * KV_HEADS, DIM))
        q, k, v = qkv.split((HEADS, KV_HEADS, KV_HEADS), dim=1)  # parts of one projection's rows
        q, k = self.rope.apply(q, pos, k=k)
        self.cache.write(k, v, batch)
        o = self.cache.attend(q, batch)
        x = x + (o.flatten(1) @ self.w_out).float()
        return self.moe.forward(x, y=x, gamma=self.gamma, accumulate=True)  # x + experts(norm(x))


def main() -> float:
    prompts, decoded = [37, 5], 6
    g = torch.Generator("cuda:0")
    g.manual_seed(1)
    xs = [torch.randn(n + decoded, 256, device="cuda:0", generator=g) for n in prompts]
    layer = DecoderLayer(max_tokens=64, max_kv_len=64, n_seqs=2)
    layer.step(torch.cat([x[:n] for x, n in zip(xs, prompts)]), prompts)
    steps = [layer.step(torch.stack([x[n + i] for x, n in zip(xs, prompts)]), [1, 1]) for i in range(decoded)]
    one_by_one = torch.stack(steps, 1)  # [sequences, decoded, hidden]
    again = DecoderLayer(max_tokens=64, max_kv_len=64, n_seqs=2)
    whole = again.step(torch.cat(xs), [n + decoded for n in prompts])
    at, off = 0, []
    for b, n in enumerate(prompts):
        want = whole[at + n:at + n + decoded]
        off.append((one_by_one[b] - want).norm() / want.norm())
        at += n + decoded
    layer.cache.device_status()
    again.cache.device_status()
    return float(torch.stack(off).max())  # (NaN where there is one)


if __name__ == "__main__":
    print(f"decoded one by one and as a prompt: relative difference {main():.2e}")
