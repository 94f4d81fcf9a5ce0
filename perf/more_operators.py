"""The dense and the expert-grouped products around the FusedMoE layer, on real work: the cases
that are measured, their inputs, and each operator in its plain form and in 64 bits.

  linear   moe_linear          out = act(x w^T + bias) + residual, bf16 or e4m3 with block scales
  grouped  moe_grouped_linear  the same per run of rows [offsets[g], offsets[g + 1]) with w[g], times
                               a weight per row
"""
import math
import random

import torch

own = False

BLOCK = 128          # e4m3: columns per scale of a row, edge of a weight's scale block
E4M3_MAX = 448.0
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "silu_mul")


def listed():
    return [
        # the gate of a small model, one token: latency
        dict(name="linear_one", op="linear", rows=1, cols=2048, outs=256, dtype="bf16", act="none",
             bias=True, residual=False),
        # the qkv projection of four running requests, 32 + 8 + 8 heads of 128
        dict(name="linear_step", op="linear", rows=4, cols=4096, outs=6144, dtype="bf16",
             act="none", bias=False, residual=False),
        # a busy server's step: the output projection back into the residual stream
        dict(name="linear_batch", op="linear", rows=96, cols=4096, outs=4096, dtype="bf16",
             act="none", bias=False, residual=True),
        # the same qkv projection of a decode batch behind a norm that wrote e4m3
        dict(name="linear_step_fp8", op="linear", rows=16, cols=7168, outs=6144, dtype="fp8",
             act="none", bias=False, residual=False),
        # an odd chunk through a layer of odd width
        dict(name="linear_ragged", op="linear", rows=777, cols=1544, outs=5001, dtype="bf16",
             act="gelu_tanh", bias=True, residual=True),
        # a full prefill batch: the tensor cores
        dict(name="linear_prompt", op="linear", rows=8192, cols=4096, outs=6144, dtype="bf16",
             act="none", bias=False, residual=False),
        # the same with 8-bit weights of a wider model, into the residual stream
        dict(name="linear_prompt_fp8", op="linear", rows=8192, cols=7168, outs=4096, dtype="fp8",
             act="none", bias=False, residual=True),
        # a decode step's rows on a rank that holds 16 experts: gate and up with the activation
        dict(name="grouped_step", op="grouped", rows=24, cols=7168, outs=4096, groups=16,
             dtype="bf16", act="silu_mul", bias=False, weighted=False, skew=1.0, sizes_seed=31),
        # the way down of the same in 8 bits, times the routing weights
        dict(name="grouped_step_fp8", op="grouped", rows=48, cols=2048, outs=7168, groups=16,
             dtype="fp8", act="none", bias=False, weighted=True, skew=1.0, sizes_seed=32),
        # a chunk, unevenly spread over the experts
        dict(name="grouped_chunk", op="grouped", rows=1500, cols=2048, outs=7168, groups=16,
             dtype="bf16", act="none", bias=True, weighted=True, skew=1.5, sizes_seed=33),
        # a full prefill batch in 8 bits
        dict(name="grouped_prompt_fp8", op="grouped", rows=8192, cols=7168, outs=4096, groups=16,
             dtype="fp8", act="silu_mul", bias=False, weighted=False, skew=0.5, sizes_seed=34),
        # a full prefill batch through eight large experts, two per token
        dict(name="grouped_prompt", op="grouped", rows=8192, cols=4096, outs=28672, groups=8,
             dtype="bf16", act="silu_mul", bias=False, weighted=False, skew=0.3, sizes_seed=35),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes over the listed ranges, never above the largest listed work."""
    most = [work(c) for c in listed()]
    top_bytes, top_flops = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        dtype = rng.choice(["bf16", "fp8"])
        act = rng.choice(ACTS)
        cols = 128 * _log_uniform(rng, 1, 56) if dtype == "fp8" else 8 * _log_uniform(rng, 8, 896)
        if act == "silu_mul":
            step = 128 if dtype == "fp8" else 16
            outs = 2 * step * _log_uniform(rng, 1, 8192 // step)
        else:
            outs = _log_uniform(rng, 1, 8192)
        c = dict(op=rng.choice(["linear", "grouped"]), rows=_log_uniform(rng, 1, 8192), cols=cols,
                 outs=outs, dtype=dtype, act=act, bias=rng.random() < 0.4)
        if c["op"] == "linear":
            c.update(residual=rng.random() < 0.4)
        else:
            c.update(groups=_log_uniform(rng, 1, 64), weighted=rng.random() < 0.4,
                     skew=rng.choice([0.0, 0.5, 1.0, 1.5]), sizes_seed=rng.randrange(1 << 30))
            sizes = _sizes(c)
            if len(sizes) * c["cols"] * (c["outs"] + 2 * max(sizes)) > 1 << 30:
                continue
        w = work(c)
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops:
            return c


def _sizes(case):
    """Rows of each group (the same for every seed): popularity rank^-skew in random order."""
    rng = random.Random(case["sizes_seed"])
    rank = list(range(1, case["groups"] + 1))
    rng.shuffle(rank)
    picks = rng.choices(range(case["groups"]), [r ** -case["skew"] for r in rank], k=case["rows"])
    sizes = [0] * case["groups"]
    for g in picks:
        sizes[g] += 1
    return sizes


def _outs(case):
    return case["outs"] // 2 if case["act"] == "silu_mul" else case["outs"]


def work(case):
    T, K, N, out = case["rows"], case["cols"], case["outs"], _outs(case)
    used = sum(n > 0 for n in _sizes(case)) if case["op"] == "grouped" else 1
    if case["dtype"] == "fp8":
        b = T * K + used * N * K + 4 * (K // BLOCK) * (T + used * -(-N // BLOCK))
    else:
        b = 2 * T * K + 2 * used * N * K
    b += 2 * T * out + (2 * used * N if case["bias"] else 0)
    b += 2 * T * out if case.get("residual") else 0
    b += 4 * T if case.get("weighted") else 0
    return {"bytes": b, "flops": 2 * T * K * N}


# ------------------------------------------------------------------------------ inputs
def _quantized(x, dims):
    """e4m3 codes of x and the scales that its blocks (dims: the axes within a block) have."""
    s = x.abs().amax(dims, keepdim=True).clamp_min(1e-10).div(E4M3_MAX)
    return (x / s).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, K, N, G = case["rows"], case["cols"], case["outs"], case.get("groups", 1)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std)

    st = dict(case=case, x_scale=None, weight_scale=None, bias=None, residual=None, row_weight=None)
    x = randn(T, K)
    shape = (G, N, K) if case["op"] == "grouped" else (N, K)
    std = K ** -0.5
    if case["dtype"] == "fp8":
        q, s = _quantized(x.view(T, -1, BLOCK), -1)
        st["x"], st["x_scale"] = q.view(T, K), s.view(T, -1).t().contiguous()
        full = -(-N // BLOCK) * BLOCK              # blocks of the last rows are cut
        w = randn(G, full, K, std=std).view(G, full // BLOCK, BLOCK, K // BLOCK, BLOCK)
        q, s = _quantized(w, (2, 4))
        st["weight"] = q.view(torch.uint8).view(G, full, K)[:, :N].contiguous().view(
            torch.float8_e4m3fn).view(shape)
        st["weight_scale"] = s.view(*shape[:-2], full // BLOCK, K // BLOCK).contiguous()
    else:
        st["x"], st["weight"] = x.to(torch.bfloat16), randn(*shape, std=std).to(torch.bfloat16)
    if case["bias"]:
        st["bias"] = randn(*shape[:-1], std=0.5).to(torch.bfloat16)
    if case.get("residual"):
        st["residual"] = randn(T, _outs(case), std=2.0).to(torch.bfloat16)
    if case["op"] == "grouped":
        sizes = _sizes(case)
        st["most"] = max(sizes)
        st["offsets"] = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
        if case["weighted"]:
            st["row_weight"] = torch.rand(T, generator=g, device="cuda")
    return st


# ------------------------------------------------------------------------------ run
def run(state):
    case = state["case"]
    if own:
        from mixture_experts_layer_05_gb300 import binding
        scales = dict(x_scale=state["x_scale"], weight_scale=state["weight_scale"])
        if case["op"] == "linear":
            return binding.moe_linear(state["x"], state["weight"], bias=state["bias"],
                                      activation=case["act"], residual=state["residual"], **scales)
        return binding.moe_grouped_linear(state["x"], state["weight"], state["offsets"],
                                          bias=state["bias"], activation=case["act"],
                                          row_weight=state["row_weight"], **scales)
    return _plain_linear(state) if case["op"] == "linear" else _plain_grouped(state)


def _activated(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "silu_mul":
        gate, up = z.chunk(2, -1)
        return gate / (1 + torch.exp(-gate)) * up
    return z


def _plain_values(st):
    """The rows and the weights as fp32 values."""
    x, w = st["x"].float(), st["weight"].float()
    if st["x_scale"] is not None:
        x = (x.view(x.shape[0], -1, BLOCK) * st["x_scale"].t()[..., None]).view_as(x)
        rows = torch.arange(w.shape[-2], device=w.device) // BLOCK
        w = w * st["weight_scale"][..., rows, :].repeat_interleave(BLOCK, -1)
    return x, w


def _plain_linear(st):
    x, w = _plain_values(st)
    z = x @ w.t()
    if st["bias"] is not None:
        z = z + st["bias"].float()
    y = _activated(z, st["case"]["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(torch.bfloat16)


def _plain_grouped(st):
    x, w = _plain_values(st)
    off = st["offsets"].long()
    t = torch.arange(x.shape[0], device=x.device)
    group = torch.searchsorted(off, t, right=True) - 1
    # each group's rows, padded to the largest group's
    row = off[:-1, None] + torch.arange(st["most"], device=x.device)
    z = torch.matmul(x[row.clamp_max(x.shape[0] - 1)], w.transpose(-1, -2))
    z = z[group, t - off[group]]
    if st["bias"] is not None:
        z = z + st["bias"].float()[group]
    y = _activated(z, st["case"]["act"])
    if st["row_weight"] is not None:
        y = y * st["row_weight"][:, None]
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    bounds = st["offsets"].tolist() if case["op"] == "grouped" else [0, case["rows"]]
    out = torch.empty(case["rows"], _outs(case), dtype=torch.float64, device=st["x"].device)
    N, half = case["outs"], _outs(case)
    fp8 = case["dtype"] == "fp8"
    for g, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        if a == b:
            continue
        x = st["x"][a:b].double()
        one = (lambda v: v[g]) if case["op"] == "grouped" else (lambda v: v)
        z = torch.zeros(b - a, N, dtype=torch.float64, device=x.device)
        if fp8:                                    # block by block, scales behind the products
            w, ws, xs = one(st["weight"]), one(st["weight_scale"]).double(), st["x_scale"].double()
            for k in range(case["cols"] // BLOCK):
                part = x[:, k * BLOCK:(k + 1) * BLOCK] @ w[:, k * BLOCK:(k + 1) * BLOCK].double().T
                z += part * xs[k, a:b, None] * ws[:, k].repeat_interleave(BLOCK)[:N]
        else:
            for n in range(0, N, 4096):
                z[:, n:n + 4096] = x @ one(st["weight"])[n:n + 4096].double().T
        if case["bias"]:
            z = z + one(st["bias"]).double()
        act = case["act"]
        if act == "relu":
            z = torch.where(z > 0, z, 0.0)
        elif act == "silu":
            z = z * torch.sigmoid(z)
        elif act == "gelu":
            z = z * torch.special.ndtr(z)
        elif act == "gelu_tanh":
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        elif act == "silu_mul":
            z = z[:, :half] * torch.sigmoid(z[:, :half]) * z[:, half:]
        if case.get("residual"):
            z = z + st["residual"][a:b].double()
        if case.get("weighted"):
            z = z * st["row_weight"][a:b, None].double()
        out[a:b] = z
    return out
