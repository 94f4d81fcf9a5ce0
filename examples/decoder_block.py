"""One decoder block served from a paged cache: norm, qkv projection, rotary cache append, paged
attention, output projection, norm with an 8-bit output, FP8 FusedMoE layer.

    python examples/decoder_block.py            # prompts, then decode steps; prints the times

Every step runs in the package's kernels; the output projection adds the residual stream in its
epilogue. Weights are random; pages are handed out by a trivial allocator.
"""
import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_layer_05_gb300 import binding, configs, inputs  # noqa: E402


@dataclass
class Sizes:
    hidden: int = 2048
    q_heads: int = 16
    kv_heads: int = 4
    head_dim: int = 128
    page: int = 32
    pages: int = 1024
    experts: int = 32
    top_k: int = 4
    intermediate: int = 512
    max_position: int = 8192
    cache: str = "bf16"            # or "fp8"


class Sequences:
    """Page tables and lengths of the running sequences (host side) and their device copies."""

    def __init__(self, s: Sizes, count: int, device="cuda"):
        self.page, self.lens, self.device = s.page, [0] * count, device
        self.free = list(range(s.pages))[::-1]
        self.owned = [[] for _ in range(count)]
        self.width = -(-s.max_position // s.page)

    def extend(self, new):
        """Room for new[i] more tokens of sequence i; (block_table, cu_seqlens_q, kv_lens)."""
        table = torch.zeros(len(new), self.width, dtype=torch.int32)
        for i, n in enumerate(new):
            self.lens[i] += n
            while len(self.owned[i]) * self.page < self.lens[i]:
                self.owned[i].append(self.free.pop())
            table[i, :len(self.owned[i])] = torch.tensor(self.owned[i], dtype=torch.int32)
        cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
        lens = torch.tensor(self.lens, dtype=torch.int32)
        return table.to(self.device), cu.to(self.device), lens.to(self.device)


class DecoderBlock:
    def __init__(self, s: Sizes, max_tokens: int, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, std=0.02):
            return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(device)

        self.s = s
        heads = s.q_heads + 2 * s.kv_heads
        self.wqkv = weight(heads * s.head_dim, s.hidden)
        self.wo = weight(s.hidden, s.q_heads * s.head_dim)
        self.status_word = binding.alloc_workspace(256, device)    # of the projections
        self.norm1, self.norm2 = 1 + weight(s.hidden), 1 + weight(s.hidden)
        self.gate = weight(s.experts, s.hidden, std=0.05)
        scale = dict(k_scale=0.05, v_scale=0.05) if s.cache == "fp8" else {}
        self.attn = binding.PagedAttention(binding.make_attn_config(
            s.q_heads, s.kv_heads, s.head_dim, s.page, cache_dtype=s.cache, **scale), device)
        shape = (s.pages, s.page, s.kv_heads, s.head_dim)
        dtype = torch.float8_e4m3fn if s.cache == "fp8" else torch.bfloat16
        self.k_cache = torch.zeros(shape, device=device, dtype=dtype)
        self.v_cache = torch.zeros(shape, device=device, dtype=dtype)
        inv = 10000.0 ** (-torch.arange(0, s.head_dim, 2, dtype=torch.float64) / s.head_dim)
        ang = torch.arange(s.max_position, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().to(device)
        w = configs.shrink(configs.TINY, num_experts=s.experts, top_k=s.top_k,
                           hidden_size=s.hidden, intermediate_size=s.intermediate)
        q = inputs.make_fp8_weights(w, seed, device=device)
        self.moe = binding.FusedMoE(binding.config_from_workload(w, weight_quant="fp8"), q["w13_q"],
                                    q["w2_q"], max_tokens=max_tokens, w13_scale=q["w13_s"],
                                    w2_scale=q["w2_s"])

    def attend(self, x, residual, batch):
        """Attention of the batch's new tokens x [T, hidden]; (attention rows, residual stream)."""
        s = self.s
        y, res, _, _ = binding.moe_rms_norm(x, self.norm1, residual=residual)
        qkv = binding.moe_linear(y, self.wqkv, workspace=self.status_word)
        qkv = qkv.view(x.shape[0], -1, s.head_dim)
        paged = (self.k_cache, self.v_cache, *batch)
        q = self.attn.append(qkv[:, :s.q_heads], qkv[:, s.q_heads:s.q_heads + s.kv_heads],
                             qkv[:, s.q_heads + s.kv_heads:], *paged, cos_sin=self.cos_sin)
        return self.attn(q, *paged), x if res is None else res

    def __call__(self, x, residual, batch):
        """(block output, residual stream): their sum is the next block's input."""
        o, res = self.attend(x, residual, batch)
        res = binding.moe_linear(o.flatten(1), self.wo, residual=res, workspace=self.status_word)
        y, _, yq, ys = binding.moe_rms_norm(res, self.norm2, out="both")
        return self.moe(y, gate_weight=self.gate, hidden_q=yq, hidden_scale=ys), res

    def status(self):
        """Of the attention with the projections around it, and of the experts."""
        attn, projections = self.attn.device_status(), binding.moe_get_device_status(self.status_word)
        return attn or projections, self.moe.device_status()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", type=int, nargs="+", default=[500, 64, 1031, 7])
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--cache", choices=("bf16", "fp8"), default="bf16")
    a = ap.parse_args(argv)
    s = Sizes(cache=a.cache)
    block = DecoderBlock(s, max_tokens=sum(a.prompts))
    seqs = Sequences(s, len(a.prompts))
    g = torch.Generator(device="cuda").manual_seed(1)

    def tokens(n):
        return torch.randn(n, s.hidden, generator=g, device="cuda").to(torch.bfloat16)

    def timed(new):
        batch, x = seqs.extend(new), tokens(sum(new))
        torch.cuda.synchronize()
        t = time.perf_counter()
        out, _ = block(x, None, batch)
        torch.cuda.synchronize()
        assert torch.isfinite(out).all() and block.status() == (binding.OK, binding.OK)
        return (time.perf_counter() - t) * 1e6

    print(f"prompts of {a.prompts} tokens: {timed(a.prompts):.0f} us (first call)")
    steps = [timed([1] * len(a.prompts)) for _ in range(a.steps)]
    print(f"one token each: {sorted(steps)[len(steps) // 2]:.0f} us (median of {a.steps} steps)")
    chunk = [64] + [1] * (len(a.prompts) - 1)
    timed(chunk)                                   # the first loads its kernels
    print(f"a chunk of 64 for the first, one for the others: {timed(chunk):.0f} us")


if __name__ == "__main__":
    main()
