"""The decoder-block operators on the GPU against their 64-bit references: RMS norm with its
8-bit output, the cache append with rotary embedding, and paged attention. Every tolerance
counts the roundings of the operator (tests/block_cases.py)."""
import math

import pytest
import torch

from mixture_experts_layer_05_gb300 import binding, configs, inputs
from tests.block_cases import (BF16, E4M3_SUB, FP8_HALF, FP32, Paged, attention_reference,
                               norm_reference, rotate_reference)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


# ------------------------------------------------------------------------------ norm
@pytest.mark.parametrize("T,H", [(1, 8), (1, 128), (3, 136), (2, 256), (5, 384), (7, 1000),
                                 (4, 5120), (33, 7168), (300, 4096), (2, 8320), (3, 32768)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("out", ["bf16", "fp8", "both"])
def test_rms_norm(cuda_lib, T, H, residual, out):
    if out != "bf16" and H % 128:
        pytest.skip("8-bit groups are 128 columns")
    g = torch.Generator().manual_seed(T * 1000 + H)
    x, w = _rand(g, T, H), (1 + _rand(g, H, std=0.2)).to(torch.bfloat16)
    r = _rand(g, T, H, std=3.0) if residual else None
    if T > 1:
        x[1] = 0                                   # a row of zeros
        if residual:
            r[1] = 0
    h, y = norm_reference(x, r, w, 1e-6)
    got = binding.moe_rms_norm(x.to(DEV), w.to(DEV), 1e-6, out=out,
                               residual=None if r is None else r.to(DEV))
    gy, gr, gq, gs = (None if t is None else t.cpu() for t in got)
    # fp32 sum of H squares: at most 32 terms a thread in sequence, two trees of five, each
    # off by FP32; half of it reaches y; the root, the division and two products add FP32 each
    d = (0.5 * (32 + 10 + 2) + 6) * FP32
    assert (gy is None) == (out == "fp8") and (gr is None) == (not residual)
    if gy is not None:
        assert ((gy.double() - y).abs() <= (BF16 * (1 + d) + d) * y.abs()).all()
    if gr is not None:
        assert ((gr.double() - h).abs() <= (BF16 + 2 * FP32) * h.abs()).all()
    if gq is not None:
        s = (y.view(T, -1, 128).abs().amax(-1).clamp_min(1e-10) / 448).t()
        assert ((gs.double() - s).abs() <= (d + 2 * FP32) * s).all()
        deq = gq.view(torch.float8_e4m3fn).double() * gs.double().t().repeat_interleave(128, 1)
        step = s.t().repeat_interleave(128, 1)
        assert ((deq - y).abs() <= (FP8_HALF + 4 * d) * y.abs() + E4M3_SUB * (1 + d) * step).all()


def test_rms_norm_strided_rows_and_aliases(cuda_lib):
    g = torch.Generator().manual_seed(5)
    big, res = _rand(g, 9, 1024).to(DEV), _rand(g, 9, 1536).to(DEV)
    w = _rand(g, 512).to(DEV)
    x, r = big[:, 256:768], res[:, 1024:]
    a = binding.moe_rms_norm(x, w, residual=r, out="both")
    b = binding.moe_rms_norm(x.contiguous(), w, residual=r.contiguous(), out="both")
    for u, v in zip(a, b):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    rc = r.contiguous()
    y, ro, _, _ = binding.moe_rms_norm(x, w, residual=rc, residual_out=rc)     # in place
    assert ro is rc and torch.equal(rc, a[1]) and torch.equal(y, a[0])


def test_rms_norm_non_finite_rows(cuda_lib):
    x = torch.ones(4, 256, dtype=torch.bfloat16)
    x[1, 7], x[2, 200], x[3, 3] = math.nan, math.inf, -math.inf
    y, _, q, _ = binding.moe_rms_norm(x.to(DEV), x[0].to(DEV), out="both")
    y, q = y.cpu().float(), q.cpu().float()
    assert torch.isfinite(y[0]).all() and torch.isfinite(q[0]).all()
    assert y[1].isnan().all() and q[1].isnan().all()
    for row, c in ((2, 200), (3, 3)):              # inf * (1 / sqrt(inf)) = NaN, 1 * 0 = 0
        assert y[row, c].isnan() and q[row, c].isnan()
        assert (y[row, :c] == 0).all() and (y[row, c + 1:] == 0).all()


def test_binding_refuses_other_tensors(cuda_lib):
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = x[0].clone()
    bad = [dict(out="int8"), dict(residual=x[:3]), dict(residual=x.float()), dict(y=x.float()),
           dict(y=x.t().contiguous().t()), dict(residual=x, residual_out=x[:3]),
           dict(out="fp8", q=x), dict(out="fp8", scale=x.float())]
    for kw in bad:
        with pytest.raises(ValueError):
            binding.moe_rms_norm(x, w, **kw)
    for args in ((x.float(), w), (x, w[:128]), (x, w.float()), (x[:, ::2], w[:128])):
        with pytest.raises(ValueError):
            binding.moe_rms_norm(*args)
    op = binding.PagedAttention(binding.make_attn_config(4, 2, 64, 16))
    c = torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    i = torch.zeros(8, dtype=torch.int32, device=DEV)
    ok = dict(q=q, k_cache=c, v_cache=c, block_table=i[:6].view(2, 3), cu_seqlens_q=i[:3],
              kv_lens=i[:2])
    op(**ok)
    for kw in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q.transpose(1, 2)), dict(k_cache=c[:4]),
               dict(k_cache=c.float()), dict(v_cache=c.permute(0, 2, 1, 3).contiguous()
                                             .permute(0, 2, 1, 3)),
               dict(k_cache=c[..., ::2], v_cache=c[..., ::2]), dict(block_table=i[:6].view(3, 2)),
               dict(block_table=i[:6].view(2, 3).long()), dict(cu_seqlens_q=i[:2]),
               dict(kv_lens=i[:4:2]), dict(out=q[:1]), dict(lse=i[:8].view(2, 4))):
        with pytest.raises(ValueError):
            op(**{**ok, **kw})
    kv = [ok[k] for k in ("k_cache", "v_cache", "block_table", "cu_seqlens_q", "kv_lens")]
    for a in ((q, q, q), (q, q[:, :2], q[:1, :2])):
        with pytest.raises(ValueError):
            op.append(*a, *kv)
    with pytest.raises(ValueError):
        op.append(q, q[:, :2], q[:, :2], *kv, cos_sin=i.view(2, 4))
    with pytest.raises(binding.GbmoeError):        # rotary_dim not a multiple of 16
        op.append(q, q[:, :2], q[:, :2], *kv, cos_sin=torch.zeros(9, 8, device=DEV))


def test_norm_output_feeds_the_fp8_layer_format(cuda_lib):
    """q and scale have the layout of moe_quant_fp8_per_token_group: on rows whose y is exact in
    bf16 (powers of two), both give the same bytes."""
    g = torch.Generator().manual_seed(3)
    x = torch.where(torch.rand(6, 512, generator=g) < 0.5, 1.0, -1.0).to(torch.bfloat16)
    w = (2.0 ** torch.randint(-6, 6, (512,), generator=g)).to(torch.bfloat16).to(DEV)
    y, _, q, s = binding.moe_rms_norm(x.to(DEV), w, 0.0, out="both")
    q2, s2 = binding.moe_quant_fp8_per_token_group(y)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("shared", [0, 128])
@pytest.mark.parametrize("gate", [False, True])
def test_fp8_layer_takes_quantized_input(cuda_lib, T, shared, gate):
    """The layer's own codes and scales, passed in, give its own result bit for bit; then the
    norm's, whose codes are of the same rows, without the hidden states' bf16 values."""
    w = configs.shrink(configs.DSV3, num_experts=16, top_k=4, num_expert_group=4, topk_group=2,
                       hidden_size=512, intermediate_size=256, shared_intermediate_size=shared)
    q = {k: None if v is None else v.to(DEV) for k, v in inputs.make_fp8_weights(w, 0).items()}
    layer = binding.FusedMoE(binding.config_from_workload(w, weight_quant="fp8"), q["w13_q"],
                             q["w2_q"], q["bias"], q["shared_w13_q"], q["shared_w2_q"],
                             max_tokens=T, w13_scale=q["w13_s"], w2_scale=q["w2_s"],
                             shared_w13_scale=q["shared_w13_s"], shared_w2_scale=q["shared_w2_s"])
    g = torch.Generator().manual_seed(T)
    x = _rand(g, T, 512).to(DEV)
    how = (dict(gate_weight=_rand(g, 16, 512, std=0.1).to(DEV)) if gate
           else dict(router_logits=torch.randn(T, 16, generator=g).to(DEV)))
    want = layer(x, **how)
    xq, xs = binding.moe_quant_fp8_per_token_group(x)
    assert torch.equal(layer(x, hidden_q=xq, hidden_scale=xs, **how), want)
    weight = (1 + _rand(g, 512, std=0.1)).to(torch.bfloat16).to(DEV)
    y, _, yq, ys = binding.moe_rms_norm(x, weight, out="both")
    rows = y if gate else torch.full_like(y, math.nan)     # only the router GEMM reads them
    out = layer(rows, hidden_q=yq, hidden_scale=ys, **how)
    assert torch.isfinite(out).all() and layer.device_status() == binding.OK
    with pytest.raises(ValueError):
        layer(x, hidden_q=xq, **how)
    with pytest.raises(ValueError):
        layer(x, hidden_q=xq, hidden_scale=xs.t().contiguous() if T != 4 else xs[:1], **how)


# ------------------------------------------------------------------------------ append
def _tables(max_pos, R):
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv,d,page,R,inter", [
    (8, 2, 64, 16, 64, False), (8, 2, 64, 8, 32, True), (7, 1, 128, 64, 128, False),
    (4, 4, 128, 32, 16, True), (32, 8, 128, 1024, 0, False)])
def test_kv_append(cuda_lib, cache, hq, hkv, d, page, R, inter):
    seqs = [(1, 1), (1, 40), (0, 9), (17, 17), (5, 130), (33, 64)]
    ks, vs = (0.03, 0.01) if cache == "fp8" else (1.0, 1.0)
    p = Paged(seqs, hkv, d, page, cache, seed=hq + d, k_scale=ks, v_scale=vs)
    qkv = _rand(p.gen, p.T, hq + 2 * hkv, d)
    cs = _tables(130, R) if R else None
    cfg = binding.make_attn_config(hq, hkv, d, page, cache_dtype=cache, k_scale=ks, v_scale=vs)
    op = binding.PagedAttention(cfg)
    kc, vc = p.shaped(p.k).to(DEV), p.shaped(p.v).to(DEV)
    x = qkv.to(DEV)
    q = op.append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, p.table.to(DEV),
                  p.cu.to(DEV), p.kv_lens.to(DEV), cos_sin=None if cs is None else cs.to(DEV),
                  interleaved=inter)
    assert op.device_status() == binding.OK
    got = {"k": kc.cpu().view(p.k.shape), "v": vc.cpu().view(p.v.shape)}
    written = torch.zeros(p.num_pages * page, dtype=torch.bool)
    for s, (n, L) in enumerate(seqs):
        t = slice(int(p.cu[s]), int(p.cu[s + 1]))
        rows = p.rows[s][L - n:]
        written[rows] = True
        want = {"q": qkv[t, :hq], "k": qkv[t, hq:hq + hkv], "v": qkv[t, hq + hkv:]}
        for name, raw in want.items():
            if R and name != "v":
                ref, size = rotate_reference(raw, cs[L - n:L, :R // 2], cs[L - n:L, R // 2:], inter)
            else:
                ref, size = raw.double(), torch.zeros(raw.shape, dtype=torch.float64)
            fp = 2 * FP32 * size                   # two products and a sum in fp32
            if name == "q" or cache == "bf16":
                have = q.cpu()[t].double() if name == "q" else got[name][rows].double()
                assert ((have - ref).abs() <= BF16 * ref.abs() + 2 * fp).all()
            else:
                sc = ks if name == "k" else vs
                have = got[name][rows].view(torch.float8_e4m3fn).double() * sc
                top = ref.clamp(-448 * sc, 448 * sc)
                assert ((have - top).abs() <= (FP8_HALF + 2 * FP32) * top.abs()
                        + E4M3_SUB * sc + 2 * fp).all()
    for name, before in (("k", p.k), ("v", p.v)):  # nothing else changed
        assert torch.equal(got[name][~written].view(torch.uint8), before[~written].view(torch.uint8))


def test_kv_append_of_huge_values(cuda_lib):
    """Quotients that leave fp32 saturate; NaN stays NaN."""
    op = binding.PagedAttention(binding.make_attn_config(1, 1, 64, 8, cache_dtype="fp8",
                                                         k_scale=1e-3, v_scale=2.0))
    x = torch.zeros(1, 1, 64)
    x[0, 0, :6] = torch.tensor([3e38, -3e38, math.inf, -math.inf, math.nan, 0.25])
    x = x.to(torch.bfloat16).to(DEV)
    i = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    k, v = (torch.zeros(1, 8, 1, 64, device=DEV, dtype=torch.float8_e4m3fn) for _ in range(2))
    op.append(x, x, x, k, v, i[:1].view(1, 1), i, i[1:])
    for c, last in ((k, 256.0), (v, 0.125)):       # 250 rounds to 256
        got = c[0, 0, 0, :6].float().cpu()
        assert got[:4].tolist() == [448.0, -448.0, 448.0, -448.0]
        assert got[4].isnan() and got[5] == last


def test_kv_append_saturates_and_works_in_place(cuda_lib):
    p = Paged([(4, 4)], 1, 64, 8, "fp8", k_scale=1.0, v_scale=1.0)
    q = torch.full((4, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    k = torch.full((4, 1, 64), 1e4, dtype=torch.bfloat16, device=DEV)
    op = binding.PagedAttention(binding.make_attn_config(2, 1, 64, 8, cache_dtype="fp8"))
    kc, vc = p.shaped(p.k).to(DEV), p.shaped(p.v).to(DEV)
    cs = _tables(4, 64).to(DEV)
    want = op.append(q, k, -k, kc, vc, p.table.to(DEV), p.cu.to(DEV), p.kv_lens.to(DEV),
                     cos_sin=cs)
    got = op.append(q, k, -k, kc, vc, p.table.to(DEV), p.cu.to(DEV), p.kv_lens.to(DEV),
                    cos_sin=cs, q_out=q)
    assert got is q and torch.equal(got, want)
    v = vc.cpu().view(p.v.shape)[p.rows[0]].view(torch.float8_e4m3fn).float()
    assert (v == -448).all()


# ------------------------------------------------------------------------------ attention
def _run(p, q, hq, causal=True, window=0, lse=True, layout="rows", stream=None, scale=None):
    cfg = binding.make_attn_config(hq, p.hkv, p.d, p.page, cache_dtype=p.cache, causal=causal,
                                   window=window, k_scale=p.k_scale, v_scale=p.v_scale,
                                   softmax_scale=scale)
    op = binding.PagedAttention(cfg)
    k, v = p.shaped(p.k).to(DEV), p.shaped(p.v).to(DEV)
    if layout == "heads":                          # [pages, heads, rows, d] in memory
        k, v = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (k, v))
    elif layout == "pair":                         # k and v pages next to each other
        both = torch.stack([k, v], 1)
        k, v = both[:, 0], both[:, 1]
    r = op(q, k, v, p.table.to(DEV), p.cu.to(DEV), p.kv_lens.to(DEV), lse=lse, stream=stream)
    torch.cuda.synchronize()
    assert op.device_status() == binding.OK
    return r


def _check(p, q, hq, causal=True, window=0, layout="rows", scale=None):
    out, lse = _run(p, q.to(DEV), hq, causal, window, layout=layout, scale=scale)
    ref, rl, bound, lb = attention_reference(p, q, causal, window, scale)
    out, lse = out.cpu().double(), lse.cpu().double()
    empty = rl == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    assert torch.isfinite(out).all()
    assert ((lse - rl).abs()[~empty] <= lb[~empty]).all()
    worst = ((out - ref).abs() / bound.clamp_min(1e-30)).max()
    assert worst <= 1.0, float(worst)


STEP = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 127), (1, 128), (1, 129), (1, 700),
        (0, 33), (1, 0), (1, 1025)]
MIXED = [(1, 1), (3, 3), (1, 300), (17, 17), (0, 5), (130, 130), (5, 4), (64, 400), (2, 0),
         (257, 300), (1, 128), (31, 129)]
HEADS = [(8, 2, 64), (4, 4, 128), (7, 1, 128), (32, 8, 128), (20, 1, 64)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("cache,page", [("bf16", 16), ("bf16", 128), ("fp8", 8), ("fp8", 64)])
@pytest.mark.parametrize("seqs", [STEP, MIXED], ids=["step", "mixed"])
def test_paged_attention(cuda_lib, hq, hkv, d, cache, page, seqs):
    ks, vs = (0.02, 0.5) if cache == "fp8" else (1.0, 1.0)
    p = Paged(seqs, hkv, d, page, cache, seed=hq * d + page, k_scale=ks, v_scale=vs)
    _check(p, _rand(p.gen, p.T, hq, d, std=1.5), hq)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 16), (True, 129),
                                           (True, 1000), (False, 50)])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("seqs", [STEP, MIXED], ids=["step", "mixed"])
def test_paged_attention_masks(cuda_lib, causal, window, cache, seqs):
    p = Paged(seqs, 2, 64, 16, cache, seed=window)
    _check(p, _rand(p.gen, p.T, 8, 64), 8, causal, window)


@pytest.mark.parametrize("layout", ["rows", "heads", "pair"])
@pytest.mark.parametrize("seqs", [STEP, MIXED], ids=["step", "mixed"])
def test_paged_attention_layouts(cuda_lib, layout, seqs):
    p = Paged(seqs, 2, 128, 32, seed=9)
    qkv = _rand(p.gen, p.T, 6 + 2 + 2, 128).to(DEV)
    q = qkv[:, 2:8]                                # rows strided
    out, lse = _run(p, q, 6, layout=layout)
    want, wl = _run(p, q.contiguous(), 6)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    _check(p, q.cpu(), 6, layout=layout)


def test_paged_attention_peaked_and_growing_scores(cuda_lib):
    """Scores whose maximum moves far from tile to tile, and one key that takes all weight."""
    p = Paged([(1, 900), (40, 700), (200, 513)], 1, 128, 16, seed=4)
    for r in p.rows:                               # k grows along the sequence
        x = p.k[r].float() * torch.linspace(0.05, 6.0, len(r))[:, None, None]
        p.k[r] = x.to(torch.bfloat16)
    q = _rand(p.gen, p.T, 8, 128, std=2.0)
    _check(p, q, 8)
    q[:, 3] = 0                                    # equal weights
    _check(p, q, 8, scale=0.7)


def test_paged_attention_long_context(cuda_lib):
    p = Paged([(1, 40001), (3, 9000), (1, 17)], 2, 128, 64, seed=8)
    _check(p, _rand(p.gen, p.T, 8, 128), 8)
    p = Paged([(70, 20011)], 1, 64, 16, "fp8", seed=8, k_scale=0.02, v_scale=0.02)
    _check(p, _rand(p.gen, p.T, 4, 64), 4)


@pytest.mark.parametrize("hq,hkv,d,cache", [(32, 8, 64, "bf16"), (12, 12, 128, "bf16"),
                                            (28, 4, 128, "fp8")])
def test_paged_attention_packed_prompts(cuda_lib, hq, hkv, d, cache):
    """Units of one and of two halves after each other in every order, several to an SM."""
    p = Paged([(1, 1), (700, 700), (33, 33), (1300, 1300), (5, 900), (100, 100), (1, 2000),
               (400, 1100), (17, 17), (2, 2)], hkv, d, 16, cache, seed=12)
    _check(p, _rand(p.gen, p.T, hq, d, std=1.5), hq)


MANY = {"prompts": [(700, 700), (1, 1)] * 2 + [(1, 9 + 30 * i) for i in range(40)] + [(1300, 1400)],
        "steps": [(1 + i % 2, 5 + 7 * i % 400) for i in range(99)] + [(60, 200), (0, 4), (1, 0)],
        "thousand": [(1, 3 + i % 140) for i in range(1100)] + [(300, 310), (1, 2)]}


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("what", list(MANY))
def test_paged_attention_many_sequences(cuda_lib, what, cache):
    """More sequences than one warp lays out, some of many row blocks, on either kernel."""
    p = Paged(MANY[what], 2, 64, 16, cache, seed=len(what))
    _check(p, _rand(p.gen, p.T, 8, 64), 8)


def test_paged_attention_offsets_past_32_bits(cuda_lib):
    """Pages beyond 2^31 elements of the cache."""
    p = Paged([(1, 200), (150, 333)], 8, 128, 128, seed=2)
    per = p.page * p.hkv * p.d
    far = 2 ** 31 // per + 1000
    big = [torch.empty(far + p.num_pages, p.page, p.hkv, p.d, dtype=torch.bfloat16, device=DEV)
           for _ in range(2)]
    for b, c in zip(big, (p.k, p.v)):
        b[far:] = p.shaped(c).to(DEV)
    q = _rand(p.gen, p.T, 8, 128)
    cfg = binding.make_attn_config(8, 8, 128, 128)
    op = binding.PagedAttention(cfg)
    table = torch.where(p.table < p.num_pages, p.table + far, p.table).to(DEV)
    out = op(q.to(DEV), *big, table, p.cu.to(DEV), p.kv_lens.to(DEV))
    want, _ = _run(p, q.to(DEV), 8)
    assert op.device_status() == binding.OK and torch.equal(out, want)


@pytest.mark.parametrize("seqs", [STEP, MIXED], ids=["step", "mixed"])
def test_paged_attention_repeats_and_streams(cuda_lib, seqs):
    """The same bits every time, on another stream too, and from a captured graph that replays
    with changed lengths."""
    p = Paged(seqs, 2, 128, 16, seed=6)
    q = _rand(p.gen, p.T, 8, 128).to(DEV)
    want, wl = _run(p, q, 8)
    for _ in range(3):
        out, lse = _run(p, q, 8)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, _ = _run(p, q, 8, stream=s)
    assert torch.equal(out, want)
    op = binding.PagedAttention(binding.make_attn_config(8, 2, 128, 16))
    args = (p.shaped(p.k).to(DEV), p.shaped(p.v).to(DEV), p.table.to(DEV), p.cu.to(DEV))
    lens = p.kv_lens.to(DEV)
    out = torch.empty_like(want)
    with torch.cuda.stream(s):
        op(q, *args, lens, out=out, stream=s)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            op(q, *args, lens, out=out)
        out.zero_()
        g.replay()
        s.synchronize()
        assert torch.equal(out, want)
        short = [(n, max(n, L - 3) if L > n else L) for n, L in seqs]
        lens.copy_(torch.tensor([L for _, L in short], dtype=torch.int32))
        g.replay()
        s.synchronize()
    p.seqs, p.kv_lens = short, lens.cpu()
    p.rows = [r[:L] for r, (_, L) in zip(p.rows, short)]
    again, _ = _run(p, q, 8)
    assert torch.equal(out, again)


def test_bad_pages_and_lengths_are_reported(cuda_lib):
    """Page ids, lengths and offsets outside their buffers: the status word says so, the other
    sequences keep their results."""
    seqs = [(1, 40), (20, 50), (1, 33), (2, 20)]
    p = Paged(seqs, 1, 64, 16, seed=1)
    q = _rand(p.gen, p.T, 4, 64).to(DEV)
    want, _ = _run(p, q, 4)
    op = binding.PagedAttention(binding.make_attn_config(4, 1, 64, 16))
    k, v = p.shaped(p.k).to(DEV), p.shaped(p.v).to(DEV)
    for what in ("page", "length", "negative"):
        table, lens = p.table.clone(), p.kv_lens.clone()
        if what == "page":
            table[1, 2], table[2, 0] = p.num_pages, -5
        elif what == "length":
            lens[1] = 16 * table.shape[1] + 1
            table[1] = table[0, 0]
        else:
            lens[1] = -4
        out = op(q, k, v, table.to(DEV), p.cu.to(DEV), lens.to(DEV))
        assert op.device_status() == binding.ERR_DEVICE_CHECK, what
        assert op.device_status() == binding.OK
        assert torch.equal(out[:1], want[:1])
        assert torch.equal(out[-2:], want[-2:])
    x = torch.zeros(p.T, 1, 64, dtype=torch.bfloat16, device=DEV)
    table = p.table.clone()
    table[3, 1] = p.num_pages
    op.append(q, x, x, k, v, table.to(DEV), p.cu.to(DEV), p.kv_lens.to(DEV))
    assert op.device_status() == binding.ERR_DEVICE_CHECK
    op.append(q, x, x, k, v, p.table.to(DEV), p.cu.to(DEV), p.kv_lens.to(DEV),
              cos_sin=_tables(10, 64).to(DEV))     # positions past the angle table
    assert op.device_status() == binding.ERR_DEVICE_CHECK


@pytest.mark.parametrize("S, T, keys", [(1024, 512, 100), (1024, 512, 1 << 24), (32, 128, 100),
                                        (32, 128, 1 << 29)])
def test_bounds_that_go_back_end_and_are_reported(cuda_lib, S, T, keys):
    """Every other sequence claims all tokens; with so many keys each that their tiles do not fit
    32 bits, which the host cannot know, the call ends without work."""
    page, width = 1024, max(1, keys // 1024)
    op = binding.PagedAttention(binding.make_attn_config(4, 1, 64, page))
    k = torch.zeros(2, page, 1, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(S, width, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T] * (S // 2) + [0], dtype=torch.int32, device=DEV)
    lens = torch.full((S,), keys, dtype=torch.int32, device=DEV)
    q = torch.zeros(T, 4, 64, dtype=torch.bfloat16, device=DEV)
    op(q, k, k, table, cu, lens)
    assert op.device_status() == binding.ERR_DEVICE_CHECK
    good = torch.arange(S + 1, dtype=torch.int32).clamp(max=T).to(DEV)
    out = op(q, k, k, table, good, torch.full_like(lens, 100))
    assert op.device_status() == binding.OK and (out == 0).all()


def _pool_of(t):
    """The stream that the allocator orders the reuse of t's memory by."""
    at = t.data_ptr()
    return [s["stream"] for s in torch.cuda.memory_snapshot()
            if s["address"] <= at < s["address"] + s["total_size"]]


@pytest.mark.parametrize("explicit", [False, True])
def test_new_outputs_belong_to_the_stream_that_writes_them(cuda_lib, explicit):
    """An output made by a call on another stream than the current one comes from that stream's
    memory: a block of the current stream's may still be in use by what is queued there."""
    g = torch.Generator().manual_seed(21)
    x, w = _rand(g, 5, 256).to(DEV), _rand(g, 256).to(DEV)
    p = Paged([(1, 20), (4, 9)], 2, 64, 16, seed=3)
    qkv = _rand(p.gen, p.T, 8, 64).to(DEV)
    k, v = p.shaped(p.k).to(DEV), p.shaped(p.v).to(DEV)
    kv = (k, v, p.table.to(DEV), p.cu.to(DEV), p.kv_lens.to(DEV))
    op = binding.PagedAttention(binding.make_attn_config(4, 2, 64, 16))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    how = dict(stream=s) if explicit else {}
    before = torch.cuda.current_stream()

    def calls(how):
        norm = binding.moe_rms_norm(x, w, residual=x, out="both", **how)
        q = op.append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], *kv, **how)
        return [*norm, q, *op(qkv[:, :4], *kv, lse=True, **how)]

    got = calls(how)
    torch.cuda.synchronize()
    want = (s if explicit else before).cuda_stream
    assert all(_pool_of(t) == [want] for t in got)
    assert torch.cuda.current_stream() == before
    for a, b in zip(got, calls({})):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    given = torch.empty(p.T, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert op(qkv[:, :4], *kv, out=given, **how) is given
    torch.cuda.synchronize()
    assert torch.equal(given, got[5])


@pytest.mark.parametrize("seqs", [[(3, 1), (1, 30)], [(9, 4), (1, 3), (40, 17)]],
                         ids=["step", "mixed"])
@pytest.mark.parametrize("causal", [True, False])
def test_paged_attention_widest_window(cuda_lib, seqs, causal):
    """A window of 2^31 - 1 is none, for tokens before position 0 too."""
    p = Paged(seqs, 2, 64, 16, seed=17)
    _check(p, _rand(p.gen, p.T, 8, 64), 8, causal, 2 ** 31 - 1)


def test_paged_attention_long_prompt(cuda_lib):
    """One prompt of 131,072 tokens, whose line in units of 8 rows would not fit 32 bits; some of
    its rows, each against a single token at its place."""
    N, at = 1 << 17, [0, 300, 65535, 131071]
    p = Paged([(N, N)], 1, 128, 64, seed=33, spare=0)
    g = torch.Generator(device=DEV).manual_seed(34)
    q = torch.randn(N, 32, 128, generator=g, device=DEV, dtype=torch.bfloat16)
    out, lse = _run(p, q, 32)
    p.seqs, p.rows = [(1, i + 1) for i in at], [p.rows[0][:i + 1] for i in at]
    p.cu = torch.arange(len(at) + 1).int()
    ref, rl, bound, lb = attention_reference(p, q[at].cpu())
    assert ((out[at].cpu().double() - ref).abs() <= bound).all()
    assert ((lse[at].cpu().double() - rl).abs() <= lb).all()


def test_paged_attention_wide_block_tables(cuda_lib):
    """Tables far wider than the sequences need: the same bits as with narrow ones. With heads of
    64, 17 rows a sequence and 8,000,000 positions a table row the units of 256 rows do not fit 32
    bits, and those of 8 rows run."""
    p = Paged([(700, 900), (1, 40)], 2, 128, 64, seed=35)
    q = _rand(p.gen, p.T, 8, 128).to(DEV)
    want, wl = _run(p, q, 8)
    p.table = torch.nn.functional.pad(p.table, (0, (1 << 14) - p.table.shape[1]), value=-1)
    out, lse = _run(p, q, 8)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    p = Paged([(17, 17 + 3 * i) for i in range(100)], 64, 64, 64, seed=36)
    p.table = torch.nn.functional.pad(p.table, (0, 62900 * 2 - p.table.shape[1]), value=-1)
    _check(p, _rand(p.gen, p.T, 64, 64), 64)


@pytest.mark.parametrize("T", [1, 2, 40], ids=["units8", "units16", "units256"])
@pytest.mark.parametrize("cache,d", [("fp8", 64), ("fp8", 128), ("bf16", 128)])
@pytest.mark.parametrize("gap", [17.5, 15.5])
@pytest.mark.parametrize("place,S", [(0, 1), (70000, 1), (150000, 1), (0, 160)])
def test_paged_attention_keeps_the_tail_of_a_peaked_row(cuda_lib, T, cache, d, gap, place, S):
    """One key lies `gap` nats above 150,000 others, whose v is 1: the columns where its own v is 0
    hold the others' share of the weight, below 1 % of the sum. One sequence, cut over all SMs, or
    160 on the same pages, most of them whole."""
    N, page = 150001, 64
    pages = -(-N // page)
    dtype = torch.float8_e4m3fn if cache == "fp8" else torch.bfloat16
    k = torch.zeros(pages * page, 1, d, device=DEV)
    v = torch.ones(pages * page, 1, d, device=DEV)
    k[place, 0, 0] = 16.0
    v[place, 0, :d // 2] = 0
    k, v = (x.to(dtype).view(pages, page, 1, d) for x in (k, v))
    cfg = binding.make_attn_config(8, 1, d, page, cache_dtype=cache, causal=False,
                                   softmax_scale=gap / 16)
    op = binding.PagedAttention(cfg)
    q = torch.zeros(S * T, 8, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1
    i32 = dict(dtype=torch.int32, device=DEV)
    out = op(q, k, v, torch.arange(pages, **i32).repeat(S, 1), torch.arange(S + 1, **i32) * T,
             torch.full((S,), N, **i32))
    assert op.device_status() == binding.OK
    tail = (N - 1) * math.exp(-cfg.softmax_scale * 16)
    share = tail / (1 + tail)
    # every weight of the tail is the same value, rounded the same way: bf16 by 2^-8 of itself; f16
    # by 2^-11, or below its normal range by 2^-25 where the largest weight is 2^10 (2^7 in units of
    # 256 rows) or more. The exponent (of at most 26, three roundings) and ex2 leave 2^-18, the fp32
    # sums at most 2^-13 when a piece has fewer than 1100 keys and there are 152, 2^-10 when it has
    # all, added 16 at a time. Then the output's rounding.
    w = BF16 if cache == "bf16" else max(2.0 ** -11, 2.0 ** (-32 if T == 40 else -35) * math.exp(gap))
    rel = w + (2.0 ** -13 if S == 1 else 2.0 ** -10) + 2.0 ** -18
    tol = torch.tensor([share * (rel + BF16 * (1 + rel)), 2.0 ** -8 + rel]).to(DEV)
    got = out.double()
    assert ((got[..., :d // 2] - share).abs() <= tol[0]).all()
    assert ((got[..., d // 2:] - 1).abs() <= tol[1]).all()


DRAFTS = {"two": [(2, 2), (2, 127), (2, 128), (2, 129), (2, 700), (2, 1), (2, 0), (2, 1026)],
          "four": [(4, 4), (4, 131), (4, 128), (4, 129), (4, 1300), (0, 7), (4, 2), (3, 400),
                   (4, 257)]}


@pytest.mark.parametrize("hq,hkv,what", [(16, 2, "two"), (8, 1, "two"), (8, 2, "four")])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 130), (False, 0)])
def test_paged_attention_drafts(cuda_lib, hq, hkv, what, cache, causal, window):
    """Two to four tokens a sequence: units of 16 rows of heads of 128."""
    seqs = DRAFTS[what]
    ks, vs = (0.02, 0.5) if cache == "fp8" else (1.0, 1.0)
    p = Paged(seqs, hkv, 128, 16, cache, seed=hq + window, k_scale=ks, v_scale=vs)
    assert 8 * len(seqs) < p.T * (hq // hkv) <= 16 * len(seqs)
    _check(p, _rand(p.gen, p.T, hq, 128, std=1.5), hq, causal, window)


@pytest.mark.parametrize("page", [8, 256, 1024])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("seqs", [STEP, DRAFTS["four"], MIXED], ids=["step", "drafts", "mixed"])
def test_paged_attention_page_sizes(cuda_lib, page, d, cache, seqs):
    """The smallest pages (32 boxes a tile) and pages of several tiles, in all units."""
    ks, vs = (0.02, 0.5) if cache == "fp8" else (1.0, 1.0)
    p = Paged(seqs, 2, d, page, cache, seed=page + d, k_scale=ks, v_scale=vs)
    _check(p, _rand(p.gen, p.T, 8, d, std=1.5), 8)


@pytest.mark.parametrize("H", [128, 1000, 4096, 7168, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_of_many_rows(cuda_lib, H, residual):
    """More than two rows an SM (two vectors a thread), and one row fewer."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(H)
    out = "bf16" if H % 128 else "both"
    for T in (2 * sms, 2 * sms + 1):
        x, w = _rand(g, T, H), (1 + _rand(g, H, std=0.2)).to(torch.bfloat16)
        r = _rand(g, T, H, std=3.0) if residual else None
        h, y = norm_reference(x, r, w, 1e-6)
        gy, gr, gq, gs = (None if t is None else t.cpu() for t in binding.moe_rms_norm(
            x.to(DEV), w.to(DEV), 1e-6, out=out, residual=None if r is None else r.to(DEV)))
        d = (0.5 * (32 + 10 + 2) + 6) * FP32       # as in test_rms_norm
        assert ((gy.double() - y).abs() <= (BF16 * (1 + d) + d) * y.abs()).all()
        if residual:
            assert ((gr.double() - h).abs() <= (BF16 + 2 * FP32) * h.abs()).all()
        if gq is not None:
            s = (y.view(T, -1, 128).abs().amax(-1).clamp_min(1e-10) / 448).t()
            assert ((gs.double() - s).abs() <= (d + 2 * FP32) * s).all()
            step = gs.double().t().repeat_interleave(128, 1)
            deq = gq.view(torch.float8_e4m3fn).double() * step
            assert ((deq - y).abs() <= (FP8_HALF + 4 * d) * y.abs()
                    + E4M3_SUB * (1 + d) * step).all()


def test_a_new_layer_serves_any_stream(cuda_lib):
    """The workspace is ready when PagedAttention returns: a first call on a stream that does not
    wait for the current one, which is busy, counts from zero."""
    p = Paged([(1, 30000), (1, 12)], 2, 64, 16, seed=41)
    q = _rand(p.gen, p.T, 8, 64).to(DEV)
    want, _ = _run(p, q, 8)
    args = (p.shaped(p.k).to(DEV), p.shaped(p.v).to(DEV), p.table.to(DEV), p.cu.to(DEV),
            p.kv_lens.to(DEV))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for fill in (0x00, 0x01, 0xFF):
        junk = torch.full((1 << 26,), fill, dtype=torch.uint8, device=DEV)   # what blocks held before
        torch.cuda.synchronize()
        del junk
        busy = torch.cuda.Event()
        torch.cuda._sleep(100_000_000)             # some 50 ms
        busy.record()
        op = binding.PagedAttention(binding.make_attn_config(8, 2, 64, 16))
        assert busy.query()                        # the zeros queued behind it are written
        out = op(q, *args, stream=s)
        s.synchronize()
        assert torch.equal(out, want) and op.device_status() == binding.OK
