"""The decoder-block operators around the FusedMoE layer, on real work: the cases that are
measured, their inputs, and each operator in its plain form and in 64 bits.

  norm    moe_rms_norm         residual addition, RMS norm, bf16 and / or e4m3 + group scales
  append  moe_kv_append        rotary embedding of new tokens, k and v into a paged cache
  attn    moe_paged_attention  attention of each sequence's new tokens over its paged cache
"""
import math
import random

import torch

own = False

GROUP = 128          # columns per scale of an 8-bit norm output
E4M3_MAX = 448.0
EPS = 1e-6
HEADS = ((32, 8, 128), (28, 4, 128), (64, 8, 64), (8, 8, 128), (16, 1, 64), (40, 8, 128))


def listed():
    return [
        # a decode step of four requests, in front of FP8 experts: latency
        dict(name="norm_step", op="norm", tokens=4, hidden=7168, residual=True, out="both"),
        # an odd batch in front of bf16 experts
        dict(name="norm_ragged", op="norm", tokens=777, hidden=5120, residual=True, out="bf16"),
        # a full prefill batch in front of FP8 experts: bandwidth
        dict(name="norm_prompt", op="norm", tokens=8192, hidden=7168, residual=True, out="both"),
        # the new tokens of 32 running requests into bf16 pages of 16
        dict(name="append_step", op="append", q_heads=32, kv_heads=8, head_dim=128, page=16,
             cache="bf16", seqs=32, decodes=32, new_min=1, new_max=1, ctx_min=100, ctx_max=4000,
             lens_seed=11, rotary=128, interleaved=False),
        # three packed prompts into e4m3 pages, rotary on half of each head
        dict(name="append_prompt", op="append", q_heads=32, kv_heads=8, head_dim=128, page=64,
             cache="fp8", seqs=3, decodes=0, new_min=1000, new_max=2500, ctx_min=0, ctx_max=300,
             lens_seed=12, rotary=64, interleaved=True),
        # a few short requests, one token each: latency
        dict(name="attn_step_small", op="attn", q_heads=32, kv_heads=8, head_dim=128, page=16,
             cache="bf16", seqs=3, decodes=3, new_min=1, new_max=1, ctx_min=50, ctx_max=1500,
             lens_seed=21, window=0, lse=False),
        # a busy server's decode step, ragged lengths
        dict(name="attn_step_batch", op="attn", q_heads=32, kv_heads=8, head_dim=128, page=16,
             cache="bf16", seqs=64, decodes=64, new_min=1, new_max=1, ctx_min=500, ctx_max=8000,
             lens_seed=22, window=0, lse=False),
        # few requests with very long contexts in an 8-bit cache, seven query heads per kv head
        dict(name="attn_step_long_fp8", op="attn", q_heads=28, kv_heads=4, head_dim=128, page=64,
             cache="fp8", seqs=5, decodes=5, new_min=1, new_max=1, ctx_min=30000, ctx_max=65000,
             lens_seed=23, window=0, lse=False),
        # packed prompts of different lengths
        dict(name="attn_prompts", op="attn", q_heads=32, kv_heads=8, head_dim=128, page=32,
             cache="bf16", seqs=5, decodes=1, new_min=200, new_max=2000, ctx_min=0, ctx_max=0,
             lens_seed=24, window=0, lse=True),
        # one long prompt
        dict(name="attn_prompt_long", op="attn", q_heads=32, kv_heads=8, head_dim=128, page=128,
             cache="bf16", seqs=1, decodes=0, new_min=8191, new_max=8191, ctx_min=0, ctx_max=0,
             lens_seed=25, window=0, lse=False),
        # chunked prefill: the next chunk of two requests far into their prompts
        dict(name="attn_chunk", op="attn", q_heads=32, kv_heads=8, head_dim=128, page=64,
             cache="bf16", seqs=2, decodes=0, new_min=300, new_max=512, ctx_min=8000,
             ctx_max=16000, lens_seed=26, window=0, lse=False),
        # a chunk and running requests in one call, 8-bit cache, small heads, sliding window
        dict(name="attn_mixed_fp8", op="attn", q_heads=64, kv_heads=8, head_dim=64, page=16,
             cache="fp8", seqs=8, decodes=7, new_min=256, new_max=256, ctx_min=1500, ctx_max=4000,
             lens_seed=27, window=1024, lse=True),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes over the listed ranges, never above the largest listed work."""
    most = [work(c) for c in listed()]
    top_bytes, top_flops = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        u = rng.random()
        if u < 0.2:
            out = rng.choice(["bf16", "fp8", "both"])
            hidden = 128 * rng.randint(1, 56) if out != "bf16" else 8 * rng.randint(16, 896)
            c = dict(op="norm", tokens=_log_uniform(rng, 1, 8192), hidden=hidden,
                     residual=rng.random() < 0.7, out=out)
        else:
            hq, hkv, d = rng.choice(HEADS)
            c = dict(op="append" if u < 0.4 else "attn", q_heads=hq, kv_heads=hkv, head_dim=d,
                     page=rng.choice([16, 32, 64, 128]), cache=rng.choice(["bf16", "fp8"]),
                     lens_seed=rng.randrange(1 << 30))
            kind = rng.choice(["step", "chunk", "prompt", "mixed"])
            if kind == "step":
                seqs = _log_uniform(rng, 1, 64)
                ctx = _log_uniform(rng, 16, 65000)
                c.update(seqs=seqs, decodes=seqs, new_min=1, new_max=1, ctx_min=max(0, ctx // 3),
                         ctx_max=ctx)
            else:
                seqs = rng.randint(1, 5)
                new = _log_uniform(rng, 2, 4096)
                ctx = 0 if kind == "prompt" else _log_uniform(rng, 16, 16000)
                c.update(seqs=seqs, decodes=seqs // 2 if kind == "mixed" else 0,
                         new_min=max(1, new // 2), new_max=new, ctx_min=ctx // 2, ctx_max=ctx)
            if c["op"] == "append":
                c.update(rotary=rng.choice([d, d // 2, 0]), interleaved=rng.random() < 0.5)
            else:
                c.update(window=_log_uniform(rng, 64, 4096) if rng.random() < 0.25 else 0,
                         lse=rng.random() < 0.5)
            new_lens, kv_lens = _lens(c)
            scores = c["seqs"] * hq * max(new_lens) * max(kv_lens)
            keys = c["seqs"] * max(kv_lens) * hkv * d
            if scores > 1 << 30 or keys > 1 << 30:
                continue
        w = work(c)
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops:
            return c


def _lens(case):
    """New tokens and total lengths of the case's sequences (the same for every seed)."""
    rng = random.Random(case["lens_seed"])
    new = [1 if i < case["decodes"] else rng.randint(case["new_min"], case["new_max"])
           for i in range(case["seqs"])]
    return new, [n + rng.randint(case["ctx_min"], case["ctx_max"]) for n in new]


def _allowed(new, total, window):
    """Sum over a sequence's new tokens of the keys each attends."""
    first = total - new + 1                        # keys of the first new token, no window
    if not window:
        return new * (first + total) // 2
    return sum(min(window, first + i) for i in range(new))


def work(case):
    if case["op"] == "norm":
        T, H = case["tokens"], case["hidden"]
        b = 2 * T * H + 2 * H
        if case["residual"]:
            b += 4 * T * H
        if case["out"] != "fp8":
            b += 2 * T * H
        if case["out"] != "bf16":
            b += T * H + 4 * T * (H // GROUP)
        return {"bytes": b, "flops": 6 * T * H}
    new, total = _lens(case)
    T = sum(new)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    code = 1 if case["cache"] == "fp8" else 2
    if case["op"] == "append":
        b = 2 * T * (hq + 2 * hkv) * d + 4 * T * case["rotary"] + 2 * T * hq * d
        return {"bytes": b + 2 * T * hkv * d * code, "flops": 3 * T * (hq + hkv) * case["rotary"]}
    window = case["window"]
    keys = sum(min(t, window + n - 1) if window else t for n, t in zip(new, total))
    pairs = sum(_allowed(n, t, window) for n, t in zip(new, total))
    b = 4 * T * hq * d + 2 * keys * hkv * d * code + (4 * T * hq if case["lse"] else 0)
    return {"bytes": b, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)

    if case["op"] == "norm":
        T, H = case["tokens"], case["hidden"]
        return dict(case=case, x=randn(T, H), weight=(1 + randn(H, std=0.1)).to(torch.bfloat16),
                    residual=randn(T, H, std=3.0) if case["residual"] else None)
    new, total = _lens(case)
    S, T, ps = case["seqs"], sum(new), case["page"]
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    pages = [-(-t // ps) for t in total]
    pool = sum(pages) + 3                          # a few pages belong to nobody
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).tolist()
    table = torch.full((S, max(pages)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):                  # entries past a sequence's end stay -1
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
    st = dict(case=case, table=table.cuda(), cu=cu.cuda(),
              kv_lens=torch.tensor(total, dtype=torch.int32, device="cuda"), max_new=max(new),
              max_total=max(total), k_scale=1.0, v_scale=1.0)
    shape = (pool, ps, hkv, d)
    if case["cache"] == "fp8":
        st["k_scale"], st["v_scale"] = 0.02, 0.015

    def cache(scale, fill):
        if not fill:
            return torch.zeros(shape, device="cuda", dtype=torch.bfloat16 if scale == 1.0
                               else torch.float8_e4m3fn)
        x = torch.randn(shape, generator=g, device="cuda")
        if case["cache"] == "fp8":
            return x.div_(scale).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return x.to(torch.bfloat16)

    fill = case["op"] == "attn"
    st["k_cache"], st["v_cache"] = cache(st["k_scale"], fill), cache(st["v_scale"], fill)
    if case["op"] == "append":
        st["qkv"] = randn(T, hq + 2 * hkv, d)      # one projection's output: q | k | v per token
        R = case["rotary"]
        if R:
            inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
            ang = torch.arange(max(total), dtype=torch.float64, device="cuda")[:, None] * inv
            st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        else:
            st["cos_sin"] = None
    else:
        st["q"] = randn(T, hq, d, std=1.5)
    return st


# ------------------------------------------------------------------------------ run
def run(state):
    case = state["case"]
    if own:
        from mixture_experts_layer_05_gb300 import binding
        if case["op"] == "norm":
            y, res, q, scale = binding.moe_rms_norm(state["x"], state["weight"], EPS,
                                                    residual=state["residual"], out=case["out"])
            return {"y": y, "residual": res, "q": q, "scale": scale}
        op = state.get("op")
        if op is None:                             # a program keeps this for the layer's life
            op = state["op"] = binding.PagedAttention(binding.make_attn_config(
                case["q_heads"], case["kv_heads"], case["head_dim"], case["page"],
                cache_dtype=case["cache"], window=case.get("window", 0),
                k_scale=state["k_scale"], v_scale=state["v_scale"]))
        paged = (state["k_cache"], state["v_cache"], state["table"], state["cu"],
                 state["kv_lens"])
        if case["op"] == "append":
            hq, hkv = case["q_heads"], case["kv_heads"]
            qkv = state["qkv"]
            q = op.append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], *paged,
                          cos_sin=state["cos_sin"], interleaved=case["interleaved"])
            return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
        if case["lse"]:
            o, lse = op(state["q"], *paged, lse=True)
            return {"o": o, "lse": lse}
        return {"o": op(state["q"], *paged)}
    if case["op"] == "norm":
        return _plain_norm(state)
    return _plain_append(state) if case["op"] == "append" else _plain_attention(state)


def _plain_norm(st):
    h, out = st["x"].float(), st["case"]["out"]
    if st["residual"] is not None:
        h = h + st["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["weight"].float()
    r = {"y": y.to(torch.bfloat16) if out != "fp8" else None,
         "residual": h.to(torch.bfloat16) if st["residual"] is not None else None,
         "q": None, "scale": None}
    if out != "bf16":
        yg = y.view(y.shape[0], -1, GROUP)
        s = yg.abs().amax(-1).clamp_min(1e-10) / E4M3_MAX
        q = (yg / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
        r["q"] = q.view_as(y).to(torch.float8_e4m3fn)
        r["scale"] = s.t().contiguous()
    return r


def _token_places(st):
    """Each new token's sequence and its index among the sequence's new tokens."""
    cu = st["cu"].long()
    t = torch.arange((st["qkv"] if "qkv" in st else st["q"]).shape[0], device=cu.device)
    s = torch.searchsorted(cu, t, right=True) - 1
    return s, t - cu[s]


def _rotate(x, c, s, interleaved):
    R = 2 * c.shape[-1]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, x[..., R:]], -1)


def _plain_append(st):
    case = st["case"]
    hq, hkv, ps = case["q_heads"], case["kv_heads"], case["page"]
    x = st["qkv"].float()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    seq, i = _token_places(st)
    cu, L = st["cu"].long(), st["kv_lens"].long()
    pos = L[seq] - (cu[1:] - cu[:-1])[seq] + i
    if st["cos_sin"] is not None:
        row = st["cos_sin"][pos][:, None]
        c, s = row.chunk(2, -1)
        q, k = _rotate(q, c, s, case["interleaved"]), _rotate(k, c, s, case["interleaved"])
    page, off = st["table"][seq, pos // ps].long(), pos % ps
    for name, val, scale in (("k_cache", k, st["k_scale"]), ("v_cache", v, st["v_scale"])):
        cache = st[name]
        if case["cache"] == "fp8":
            code = (val / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[page, off] = code.view(torch.uint8)
        else:
            cache[page, off] = val.to(torch.bfloat16)
    return {"q": q.to(torch.bfloat16), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attention(st):
    case = st["case"]
    hq, hkv, d, ps = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    G, N, M = hq // hkv, st["max_new"], st["max_total"]
    cu, L = st["cu"].long(), st["kv_lens"].long()
    S, dev = L.shape[0], L.device
    n = cu[1:] - cu[:-1]
    i, j = torch.arange(N, device=dev), torch.arange(M, device=dev)
    # padded [S, kv heads, G * N queries, d] and [S, kv heads, M keys, d]
    tok = torch.minimum(cu[:-1, None] + i, cu[1:, None] - 1)
    q = st["q"].float()[tok].view(S, N, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(S, hkv, -1, d)
    page = st["table"].long()[:, j // ps].clamp_min(0)
    off = (j % ps).expand_as(page)

    def keys(cache, scale):
        if case["cache"] == "fp8":
            x = cache.view(torch.uint8)[page, off].view(torch.float8_e4m3fn).float() * scale
        else:
            x = cache[page, off].float()
        return x.permute(0, 2, 1, 3)               # [S, kv heads, M, d]

    s = torch.matmul(q, keys(st["k_cache"], st["k_scale"]).transpose(-1, -2)).mul_(d ** -0.5)
    s = s.view(S, hkv, G, N, M)
    pos = (L - n)[:, None] + i                     # [S, N]
    dead = (j > pos[..., None]) | (j >= L[:, None, None])
    if case["window"]:
        dead |= j <= pos[..., None] - case["window"]
    s.masked_fill_(dead[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, hkv, G * N, M), keys(st["v_cache"], st["v_scale"]))
    o = o.view(S, hkv, G, N, d) / total.clamp_min(torch.finfo(torch.float32).tiny)
    seq, at = _token_places(st)
    o = o.permute(0, 3, 1, 2, 4)[seq, at].reshape(-1, hq, d).to(torch.bfloat16)
    if not case["lse"]:
        return {"o": o}
    lse = (m + total.log()).squeeze(-1).permute(0, 3, 1, 2)[seq, at].reshape(-1, hq)
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double()
        if case["residual"]:
            h = h + st["residual"].double()
        y = h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / case["hidden"] + EPS)
        y = y * st["weight"].double()
        r = {"y": None if case["out"] == "fp8" else y, "residual": h if case["residual"] else None,
             "q": None, "scale": None}
        if case["out"] != "bf16":
            groups = y.split(GROUP, dim=1)
            s = torch.stack([torch.maximum(a.abs().max(1).values,
                                           torch.tensor(1e-10, device=y.device)) / E4M3_MAX
                             for a in groups])
            r["scale"] = s
            r["q"] = torch.cat([(a / b[:, None]).float().to(torch.float8_e4m3fn)
                                for a, b in zip(groups, s)], 1)
        return r
    new, total = _lens(case)
    hq, hkv, d, ps = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    table, fp8 = st["table"].tolist(), case["cache"] == "fp8"
    dev = st["kv_lens"].device
    if case["op"] == "append":
        out_q = []
        kc = st["k_cache"].to(torch.float64)
        vc = st["v_cache"].to(torch.float64)
        t0 = 0
        for s in range(case["seqs"]):
            x = st["qkv"][t0:t0 + new[s]].double()
            t0 += new[s]
            at = list(range(total[s] - new[s], total[s]))
            pos = torch.tensor(at, device=dev)
            R = case["rotary"]
            if R:
                c = st["cos_sin"][pos, :R // 2].double()
                z = st["cos_sin"][pos, R // 2:].double()
                turn = torch.complex(c, z)[:, None]            # (a + ib) e^{i angle}
                qk = x[:, :hq + hkv]
                if case["interleaved"]:
                    w = torch.view_as_complex(qk[..., :R].reshape(*qk.shape[:2], -1, 2)
                                              .contiguous()) * turn
                    r = torch.view_as_real(w).reshape(*qk.shape[:2], R)
                else:
                    w = torch.complex(qk[..., :R // 2].contiguous(),
                                      qk[..., R // 2:R].contiguous()) * turn
                    r = torch.cat([w.real, w.imag], -1)
                x[:, :hq + hkv, :R] = r
            out_q.append(x[:, :hq])
            rows = torch.tensor([table[s][p // ps] for p in at], device=dev)
            kc[rows, pos % ps] = x[:, hq:hq + hkv] / (st["k_scale"] if fp8 else 1.0)
            vc[rows, pos % ps] = x[:, hq + hkv:] / (st["v_scale"] if fp8 else 1.0)
        if fp8:
            kc, vc = (c.clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn)
                      for c in (kc, vc))
        return {"q": torch.cat(out_q), "k_cache": kc, "v_cache": vc}
    o = torch.empty(sum(new), hq, d, dtype=torch.float64, device=dev)
    lse = torch.empty(sum(new), hq, dtype=torch.float64, device=dev)
    t0 = 0
    for s in range(case["seqs"]):
        rows = torch.tensor(table[s][:-(-total[s] // ps)], device=dev)
        byte = (lambda c: c.view(torch.uint8)[rows].view(c.dtype)) if fp8 else (lambda c: c[rows])
        k = byte(st["k_cache"]).double().reshape(-1, hkv, d)[:total[s]] * st["k_scale"]
        v = byte(st["v_cache"]).double().reshape(-1, hkv, d)[:total[s]] * st["v_scale"]
        for a in range(0, new[s], 1024):           # blocks of queries
            b = min(a + 1024, new[s])
            first, last = total[s] - new[s] + a, total[s] - new[s] + b   # positions [first, last)
            lo = max(0, first - case["window"] + 1) if case["window"] else 0
            key = torch.arange(lo, last, device=dev)
            p = torch.arange(first, last, device=dev)[:, None]
            seen = key <= p
            if case["window"]:
                seen = seen & (key > p - case["window"])
            for h in range(hq):
                e = st["q"][t0 + a:t0 + b, h].double() @ k[lo:last, h // (hq // hkv)].T
                e = torch.where(seen, e / math.sqrt(d), -math.inf)
                o[t0 + a:t0 + b, h] = torch.softmax(e, -1) @ v[lo:last, h // (hq // hkv)]
                lse[t0 + a:t0 + b, h] = torch.logsumexp(e, -1)
        t0 += new[s]
    return {"o": o, "lse": lse} if case["lse"] else {"o": o}
