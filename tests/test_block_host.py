"""The decoder-block operators on the host: argument refusals of the C ABI and the binding, and
the index rules of the paged batch (csrc/paged_checks.h, compiled for the host)."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest
import torch

from mixture_experts_layer_05_gb300 import binding
from mixture_experts_layer_05_gb300 import build as build_mod

P = ctypes.c_void_p
OK, BAD, UNSUP, WS = (binding.OK, binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED,
                      binding.ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return binding.load()


def _norm(lib, T=4, H=256, x=256, xs=None, res=0, rs=0, w=256, eps=1e-6, y=256, ro=0, q=0, s=0):
    a = binding.RmsNormArgs(x or None, H if xs is None else xs, res or None, rs, w or None, eps,
                            y or None, ro or None, q or None, s or None)
    return lib.moe_rms_norm(T, H, ctypes.byref(a), None)


def test_rms_norm_refusals(lib):
    assert lib.moe_rms_norm(0, 256, None, None) == OK                  # empty batch
    assert lib.moe_rms_norm(4, 256, None, None) == BAD
    for kw in (dict(T=-1), dict(H=0), dict(x=0), dict(w=0), dict(y=0), dict(q=256), dict(s=256),
               dict(ro=256), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(x=264), dict(w=264), dict(y=264), dict(q=264, s=256), dict(q=256, s=258),
               dict(xs=128), dict(xs=260), dict(res=256, rs=128), dict(res=256, rs=260),
               dict(res=264, rs=256), dict(res=256, rs=256, ro=264)):
        assert _norm(lib, **kw) == BAD, kw
    for kw in (dict(H=100), dict(H=264, q=256, s=256), dict(H=32776)):
        assert _norm(lib, **kw) == UNSUP, kw


def _cfg(**kw):
    d = dict(num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16)
    d.update(kw)
    return binding.make_attn_config(**d)


def _kv(**kw):
    d = dict(k_cache=256, v_cache=256, page_stride=2048, token_stride=128, head_stride=64,
             num_pages=4, num_seqs=2, block_table_stride=3, block_table=256, cu_seqlens_q=256,
             kv_lens=256)
    d.update(kw)
    return binding.PagedKv(**d)


BAD_CONFIGS = (dict(num_q_heads=0), dict(num_kv_heads=0), dict(num_q_heads=9),
               dict(num_q_heads=2048), dict(head_dim=0, softmax_scale=1.0), dict(page_size=0),
               dict(window=-1), dict(cache_dtype=7), dict(softmax_scale=0.0),
               dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf")),
               dict(k_scale=0.5), dict(v_scale=2.0), dict(cache_dtype="fp8", k_scale=0.0),
               dict(cache_dtype="fp8", v_scale=float("inf")))
UNSUP_CONFIGS = (dict(head_dim=96), dict(head_dim=256), dict(page_size=4), dict(page_size=24),
                 dict(page_size=2048))
BAD_KV = (dict(k_cache=None), dict(v_cache=None), dict(block_table=None), dict(cu_seqlens_q=None),
          dict(kv_lens=None), dict(num_pages=0), dict(num_seqs=0), dict(block_table_stride=0),
          dict(page_stride=0), dict(token_stride=-64), dict(head_stride=0), dict(k_cache=264),
          dict(v_cache=264), dict(page_stride=2052), dict(token_stride=132), dict(head_stride=68),
          dict(block_table=258), dict(cu_seqlens_q=258), dict(kv_lens=258))


def _attn(lib, cfg=None, T=4, kv=None, q=256, qs=512, out=256, lse=0, ws=256, nbytes=1 << 40):
    cfg, kv = cfg or _cfg(), kv or _kv()
    return lib.moe_paged_attention(ctypes.byref(cfg), T, ctypes.byref(kv), P(q or None), qs,
                                   P(out or None), P(lse or None), P(ws or None), nbytes, None)


def test_paged_attention_refusals(lib):
    assert lib.moe_paged_attention(None, 4, None, None, 0, None, None, None, 0, None) == BAD
    assert _attn(lib, T=0) == OK
    for kw in BAD_CONFIGS:
        assert _attn(lib, cfg=_cfg(**kw)) == BAD, kw
        assert lib.moe_paged_attention_workspace_size(ctypes.byref(_cfg(**kw))) == 0, kw
    for kw in UNSUP_CONFIGS:
        assert _attn(lib, cfg=_cfg(**kw)) == UNSUP, kw
        assert lib.moe_paged_attention_workspace_size(ctypes.byref(_cfg(**kw))) == 0, kw
    for kw in BAD_KV:
        assert _attn(lib, kv=_kv(**kw)) == BAD, kw
    assert _attn(lib, kv=_kv(num_seqs=8193)) == UNSUP
    assert _attn(lib, cfg=_cfg(num_q_heads=1024), T=1 << 21, qs=65536) == UNSUP
    assert _attn(lib, T=1 << 22, kv=_kv(block_table_stride=1 << 22)) == UNSUP
    for kw in (dict(T=-1), dict(q=0), dict(out=0), dict(qs=504), dict(qs=516), dict(q=264),
               dict(out=264), dict(lse=258)):
        assert _attn(lib, **kw) == BAD, kw
    need = lib.moe_paged_attention_workspace_size(ctypes.byref(_cfg()))
    assert need >= 256
    for kw in (dict(ws=0), dict(ws=128), dict(nbytes=need - 1)):
        assert _attn(lib, **kw) == WS, kw


def _append(lib, cfg=None, T=4, kv=None, **kw):
    cfg, kv = cfg or _cfg(), kv or _kv()
    d = dict(q=256, k=256, v=256, q_stride=768, k_stride=768, v_stride=768, cos_sin=256,
             max_position=64, rotary_dim=64, interleaved=0, q_out=256, workspace=256)
    d.update(kw)
    return lib.moe_kv_append(ctypes.byref(cfg), T, ctypes.byref(kv),
                             ctypes.byref(binding.KvAppendArgs(**d)), None)


def test_kv_append_refusals(lib):
    assert lib.moe_kv_append(None, 4, None, None, None) == BAD
    assert _append(lib, T=0) == OK
    for kw in BAD_CONFIGS:
        assert _append(lib, cfg=_cfg(**kw)) == BAD, kw
    for kw in UNSUP_CONFIGS:
        assert _append(lib, cfg=_cfg(**kw)) == UNSUP, kw
    for kw in BAD_KV:
        assert _append(lib, kv=_kv(**kw)) == BAD, kw
    for kw in (dict(T=-1), dict(q=None), dict(k=None), dict(v=None), dict(q_out=None),
               dict(q_stride=504), dict(q_stride=516), dict(k_stride=120), dict(k_stride=132),
               dict(v_stride=120), dict(v_stride=132), dict(q=264), dict(k=264), dict(v=264),
               dict(q_out=264), dict(cos_sin=264), dict(workspace=128), dict(rotary_dim=80),
               dict(rotary_dim=8), dict(rotary_dim=-16), dict(rotary_dim=0), dict(cos_sin=None),
               dict(max_position=0)):
        assert _append(lib, **kw) == BAD, kw


def test_forward_q_refusals(lib):
    def call(cfg, T=4, q=256, s=256, logits=256):
        a = binding.ForwardArgs(router_logits=logits or None, w13_weight=256, w2_weight=256,
                                output=256, workspace=256, workspace_bytes=1 << 40, w13_scale=256,
                                w2_scale=256, gate_weight=None if logits else 256)
        return lib.moe_forward_q(ctypes.byref(cfg), T, ctypes.byref(a), P(q or None), P(s or None),
                                 None)
    make = lambda quant: binding.make_config(8, 2, 256, 256, weight_quant=quant)  # noqa: E731
    fp8 = make("fp8")
    assert lib.moe_forward_q(None, 4, None, None, None, None) == BAD
    assert call(make(None)) == UNSUP and call(make("nvfp4")) == UNSUP
    assert call(fp8, T=0, q=0, s=0) == OK
    for kw in (dict(T=-1), dict(q=0), dict(s=0), dict(q=264), dict(s=258),
               dict(logits=0)):                  # the router GEMM needs the hidden states
        assert call(fp8, **kw) == BAD, kw
    assert lib.moe_forward_q(ctypes.byref(fp8), 4, None, P(256), P(256), None) == BAD


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.moe_rms_norm(x, x[0])
    with pytest.raises(binding.GbmoeError):
        binding.PagedAttention(_cfg(head_dim=96), device="cpu")
    op = binding.PagedAttention(_cfg(), device="cpu")
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        op(torch.zeros(2, 8, 64, dtype=torch.bfloat16), c, c, i[None], i[:2], i[:1])


CHECKS = r"""
#include <cstdio>
#include "paged_checks.h"
using namespace gbmoe;
int main() {
  int q0, q1, L, T, n, i, causal, window, id, pages;
  long long cap;
  char kind;
  while (scanf(" %c", &kind) == 1) {
    bool bad = false;
    if (kind == 's') {
      if (scanf("%d %d %d %d %lld", &q0, &q1, &L, &T, &cap) != 5) return 1;
      const SeqInfo r = checked_seq(q0, q1, L, T, cap, &bad);
      printf("%d %d %d %d\n", r.q0, r.n, r.L, bad);
    } else if (kind == 'k') {
      if (scanf("%d %d %d %d %d", &L, &n, &i, &causal, &window) != 5) return 1;
      const KeyRange r = key_range(SeqInfo{0, n, L}, i, causal != 0, window);
      printf("%d %d\n", r.lo, r.hi);
    } else {
      if (scanf("%d %d", &id, &pages) != 2) return 1;
      printf("%d", checked_page(id, pages, &bad));
      printf(" %d\n", bad);
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def checks(tmp_path_factory):
    d = tmp_path_factory.mktemp("checks")
    (d / "checks.cpp").write_text(CHECKS)
    subprocess.run(["g++", "-std=c++17", "-I", build_mod.CSRC, str(d / "checks.cpp"), "-o",
                    str(d / "checks")], check=True)

    def ask(lines):
        out = subprocess.run([str(d / "checks")], input="\n".join(lines), text=True,
                             capture_output=True, check=True).stdout
        return [tuple(int(x) for x in l.split()) for l in out.splitlines()]
    return ask


def test_sequences_stay_in_their_buffers(checks):
    """Whatever the arrays hold, tokens lie in the batch and keys in the block table."""
    vals = (-(2 ** 31), -1, 0, 1, 5, 7, 8, 2 ** 30, 2 ** 31 - 1)
    asks = [(q0, q1, L, 7, cap) for q0, q1, L in itertools.product(vals, vals, vals)
            for cap in (8, 2 ** 30, 2 ** 41)]
    got = checks(["s " + " ".join(map(str, a)) for a in asks])
    for (q0, q1, L, T, cap), (r0, n, rL, bad) in zip(asks, got):
        assert 0 <= r0 and 0 <= n and r0 + n <= T
        assert 0 <= rL <= min(cap, 2 ** 30)
        good = 0 <= q0 <= q1 <= T and 0 <= L <= min(cap, 2 ** 30)
        assert bad == (not good)
        if good:
            assert (r0, n, rL) == (q0, q1 - q0, L)


def test_key_ranges_match_the_definition(checks):
    asks = [(L, n, i, causal, w) for L in (0, 1, 2, 5, 9) for n in (1, 3, 9) for i in range(n)
            for causal in (0, 1) for w in (0, 1, 2, 7)]
    got = checks(["k " + " ".join(map(str, a)) for a in asks])
    for (L, n, i, causal, w), (lo, hi) in zip(asks, got):
        pos = L - n + i
        want = [j for j in range(L) if (not causal or j <= pos) and (not w or j > pos - w)]
        assert list(range(lo, hi)) == want


def test_pages_stay_in_the_cache(checks):
    asks = [(i, p) for i in (-(2 ** 31), -1, 0, 3, 4, 5, 2 ** 31 - 1) for p in (1, 4, 2 ** 31 - 1)]
    got = checks([f"p {i} {p}" for i, p in asks])
    for (i, p), (page, bad) in zip(asks, got):
        assert 0 <= page < p and bad == (not 0 <= i < p)
        if not bad:
            assert page == i


PLAN = r"""
#include <cstdio>
#include <vector>
#include "attn_plan.h"
using namespace gbmoe;
struct Shape : AttnShape {
  int half, full;
};
int main() {
  Shape a;
  int causal, g, S, G;
  while (scanf("%d %d %d %d %d %d %d %d %d %d", &G, &a.hkv, &a.br_shift, &a.extra, &a.half,
               &a.full, &causal, &a.window, &g, &S) == 10) {
    a.causal = causal != 0;
    set_group(a, G);
    std::vector<SeqInfo> q(S);
    std::vector<int> line(S + 1, 0);
    for (int s = 0, q0 = 0; s < S; ++s) {
      if (scanf("%d %d", &q[s].n, &q[s].L) != 2) return 1;
      q[s].q0 = q0;
      q0 += q[s].n;
      line[s + 1] = line[s] + seq_length(a, q[s]) * a.hkv;
    }
    g = line_ctas(a, line[S], g);
    for (int c = 0; c < g; ++c) {
      const int at = range_at(line[S], c, g), end = range_at(line[S], c + 1, g);
      if (end <= at) continue;
      int s = 0;
      while (line[s + 1] <= at) ++s;
      const int head = (line[s + 1] - line[s]) / a.hkv;
      AttnCursor cur = {s, (at - line[s]) / head, 0, 0, end - at};
      walk_blocks(a, q[s], (at - line[s]) % head, cur);
      while (cur.left > 0) {
        while (q[cur.s].n == 0) ++cur.s;
        const AttnPiece p = take_piece(a, q[cur.s], cur);
        if (p.ta == p.tb) continue;
        printf("%d %d %d %d %d %d %d %d ", c, p.s, p.head, p.rb, p.ta, p.tb, p.u.t0, p.u.tiles);
      }
    }
    printf("\n");
  }
  return 0;
}
"""


def test_attention_work_is_cut_whole(tmp_path):
    """Every tile that a unit's tokens attend is computed once, the pieces of a unit follow each
    other over neighbouring CTAs, no CTA has more than its share of the cost, and a CTA begins
    at most one unit that it leaves and ends at most one that it did not begin."""
    (tmp_path / "plan.cpp").write_text(PLAN)
    subprocess.run(["g++", "-std=c++17", "-I", build_mod.CSRC, str(tmp_path / "plan.cpp"), "-o",
                    str(tmp_path / "plan")], check=True)
    rng = random.Random(7)
    cases = []
    for _ in range(300):
        S = rng.choice([1, 1, 2, 5, 12])
        seqs = []
        for _ in range(S):
            n = rng.choice([0, 1, 1, 2, 17, 64, 130, 300])
            seqs.append((n, max(0, rng.choice([n, n + 1, n - 2, n + 127, n + 128, n + 5000, 0]))))
        if not any(n for n, _ in seqs):
            seqs[0] = (1, 3)
        cases.append((rng.choice([1, 2, 3, 4, 7, 8, 20, 1024]), rng.choice([1, 2, 8]), rng.choice([4, 8]),
                      rng.choice([0, 1, 3]), *rng.choice([(1, 1), (1, 2), (4, 5)]), int(rng.random() < 0.8), rng.choice([0, 0, 1, 100, 1000]),
                      rng.choice([1, 7, 148, 152]), S, seqs))
    text = "\n".join(" ".join(map(str, c[:10])) + " " + " ".join(f"{n} {L}" for n, L in c[10])
                     for c in cases)
    out = subprocess.run([str(tmp_path / "plan")], input=text, text=True, capture_output=True,
                         check=True).stdout.splitlines()
    assert len(out) == len(cases)
    for (G, hkv, shift, extra, half, full, causal, window, g, S, seqs), line in zip(cases, out):
        BR, TK = 1 << shift, 128
        v = [int(x) for x in line.split()]
        pieces = [tuple(v[i:i + 8]) for i in range(0, len(v), 8)]
        units = {}
        for s, (n, L) in enumerate(seqs):
            for head in range(hkv):
                for rb in range(-(-n * G // BR)):
                    toks = range(rb * BR // G, (min(n * G, (rb + 1) * BR) - 1) // G + 1)
                    keys = set()
                    for i in (toks[0], toks[-1]):
                        pos = L - n + i
                        lo = max(0, pos - window + 1) if window else 0
                        hi = min(L, pos + 1) if causal else L
                        keys.add((lo, hi))
                    lo, hi = min(k[0] for k in keys), max(k[1] for k in keys)
                    units[s, head, rb] = (lo // TK, -(-hi // TK)) if hi > lo else (0, 1)
        at, per, order = {}, {}, list(units)
        cost = {(s, h, rb): full if 2 * min(BR, seqs[s][0] * G - rb * BR) > BR else half
                for s, h, rb in units}
        total = sum((b - a) * cost[u] + extra for u, (a, b) in units.items())
        g = min(g, -(-total // full))
        where = 0
        for c, s, head, rb, ta, tb, t0, tiles in pieces:
            u = (s, head, rb)
            assert units[u] == (t0, t0 + tiles)
            assert ta == at.get(u, 0) and ta < tb <= tiles
            at[u] = tb
            while order[where] != u:               # the line's order
                where += 1
            per.setdefault(c, []).append((ta > 0, tb < tiles, (tb - ta) * cost[u]))
        assert all(at[u] == b - a for u, (a, b) in units.items())
        held = {}                                  # a cut unit's CTAs are neighbours
        for c, s, head, rb, *_ in pieces:
            held.setdefault((s, head, rb), []).append(c)
        assert all(cs == list(range(cs[0], cs[-1] + 1)) for cs in held.values())
        for c, ps in per.items():
            begun = sum(not p[0] for p in ps)      # their extra cost lies in this range, but
            share = sum(p[2] for p in ps) + extra * begun      # for a cut through it at an end
            assert total / g - full - extra < share < total / g + full + extra
            assert not any(p[0] for p in ps[1:]) and not any(p[1] for p in ps[:-1])


DIVIDE = r"""
#include <cstdio>
#include "attn_plan.h"
using namespace gbmoe;
int main() {
  long bad = 0;
  for (int G = 1; G <= 1024; ++G) {
    AttnShape a;
    set_group(a, G);
    for (long r = 0; r < 5000; ++r) bad += div_group(a, (int)r) != r / G;
    for (long k = 1; k * G < 2147483647L; k = k * 3 + 1)
      for (long r = k * G - 2; r <= k * G + 2; ++r)
        if (r >= 0 && r < 2147483647L) bad += div_group(a, (int)r) != r / G;
    for (long r = 2147483600L; r < 2147483647L; ++r) bad += div_group(a, (int)r) != r / G;
  }
  printf("%ld", bad);
  return 0;
}
"""


def test_division_by_the_group_is_exact(tmp_path):
    (tmp_path / "divide.cpp").write_text(DIVIDE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build_mod.CSRC, str(tmp_path / "divide.cpp"),
                    "-o", str(tmp_path / "divide")], check=True)
    out = subprocess.run([str(tmp_path / "divide")], capture_output=True, text=True, check=True)
    assert out.stdout == "0"


def _fake(*shape, dtype=torch.bfloat16, device="cuda:0"):
    return torch.empty(*shape, dtype=dtype, device=device)


def test_binding_refuses_tensors_of_two_devices(lib):
    """Every tensor of a call is on one device (fake tensors: the checks come before any address
    is used)."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(allow_non_fake_inputs=True):
        norm = dict(x=_fake(4, 256), weight=_fake(256), residual=_fake(4, 256), out="both",
                    y=_fake(4, 256), residual_out=_fake(4, 256),
                    q=_fake(4, 256, dtype=torch.float8_e4m3fn),
                    scale=_fake(2, 4, dtype=torch.float32))
        for name in norm:
            if name in ("x", "out"):
                continue
            with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
                binding.moe_rms_norm(**{**norm, name: norm[name].to("cuda:1")})
        op = binding.PagedAttention(_cfg(), device="cuda:0")
        i32 = dict(dtype=torch.int32)
        kv = dict(k_cache=_fake(4, 16, 2, 64), v_cache=_fake(4, 16, 2, 64),
                  block_table=_fake(1, 3, **i32), cu_seqlens_q=_fake(2, **i32),
                  kv_lens=_fake(1, **i32))
        attend = dict(kv, q=_fake(2, 8, 64), out=_fake(2, 8, 64),
                      lse=_fake(2, 8, dtype=torch.float32))
        append = dict(kv, q=_fake(2, 8, 64), k=_fake(2, 2, 64), v=_fake(2, 2, 64),
                      cos_sin=_fake(9, 64, dtype=torch.float32), q_out=_fake(2, 8, 64))
        for call, good in ((op, attend), (op.append, append)):
            for name in good:
                with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
                    call(**{**good, name: good[name].to("cuda:1")})
        far = binding.PagedAttention(_cfg(), device="cuda:1")     # its workspace
        for call, good in ((far, attend), (far.append, append)):
            with pytest.raises(ValueError, match="is on cuda:0"):
                call(**good)


def test_a_flag_without_a_truth_value_raises(lib):
    from torch._subclasses.fake_tensor import FakeTensorMode

    class Unclear:
        def __bool__(self):
            raise KeyError("unclear")
    i32 = dict(dtype=torch.int32)
    with FakeTensorMode(allow_non_fake_inputs=True):
        op = binding.PagedAttention(_cfg(), device="cuda:0")
        with pytest.raises(KeyError, match="unclear"):
            op.append(_fake(2, 8, 64), _fake(2, 2, 64), _fake(2, 2, 64), _fake(4, 16, 2, 64),
                      _fake(4, 16, 2, 64), _fake(1, 3, **i32), _fake(2, **i32), _fake(1, **i32),
                      interleaved=Unclear())


def test_sizes_past_32_bits_are_refused(lib):
    """A size that the C ABI's 32 bits would cut to another one."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    far = 2 ** 32 + 4
    i32 = dict(dtype=torch.int32)
    with FakeTensorMode(allow_non_fake_inputs=True):
        with pytest.raises(ValueError, match="32 bits"):
            binding.moe_rms_norm(_fake(far, 8), _fake(8))
        with pytest.raises(ValueError, match="32 bits"):
            binding.moe_rms_norm(_fake(4, far), _fake(far))
        op = binding.PagedAttention(_cfg(), device="cuda:0")
        good = dict(k_cache=_fake(4, 16, 2, 64), v_cache=_fake(4, 16, 2, 64),
                    block_table=_fake(1, 3, **i32), cu_seqlens_q=_fake(2, **i32),
                    kv_lens=_fake(1, **i32))
        caches = dict(k_cache=_fake(far, 16, 2, 64), v_cache=_fake(far, 16, 2, 64))
        many = dict(block_table=_fake(far, 1, **i32), cu_seqlens_q=_fake(far + 1, **i32),
                    kv_lens=_fake(far, **i32))
        for kv, T in ((good, far), ({**good, **caches}, 2), ({**good, **many}, 2),
                      ({**good, "block_table": _fake(1, far, **i32)}, 2)):
            with pytest.raises(ValueError, match="32 bits"):
                op(_fake(T, 8, 64), **kv)
            with pytest.raises(ValueError, match="32 bits"):
                op.append(_fake(T, 8, 64), _fake(T, 2, 64), _fake(T, 2, 64), **kv)
        q, k = _fake(2, 8, 64), _fake(2, 2, 64)
        for shape in ((far, 16), (1, far)):
            with pytest.raises(ValueError, match="32 bits"):
                op.append(q, k, k, **good, cos_sin=_fake(*shape, dtype=torch.float32))


def test_key_ranges_of_the_widest_windows(checks):
    """Tokens before position 0 (more new tokens than keys) and a window of up to 2^31 - 1: the
    range does not leave 32 bits on its way."""
    top = 2 ** 31 - 1
    asks = [(L, n, i, causal, w) for L, n in ((0, 6), (1, 5), (3, 9), (100, 4000000), (2 ** 30, 1))
            for i in (0, 1, n // 2, n - 1) for causal in (0, 1) for w in (top, top - 1, 2 ** 30)]
    got = checks(["k " + " ".join(map(str, a)) for a in asks])
    for (L, n, i, causal, w), (lo, hi) in zip(asks, got):
        pos = L - n + i
        want = max(0, pos - w + 1), min(L, pos + 1) if causal else L
        assert (lo, hi) == want or (hi <= lo and want[1] <= want[0])


# heads, new tokens, sequences and positions of a block table row that attention takes
WIDE_CALLS = ((32, 8, 128, 131072, 1, 131072), (64, 8, 128, 98304, 1, 98304),
              (32, 8, 128, 16384, 1, 1 << 20), (32, 8, 128, 32768, 64, 1 << 20),
              (64, 64, 64, 1700, 100, 62900 * 128), (32, 8, 64, 131072, 1, 131072),
              (32, 8, 128, 1 << 20, 1, 1 << 20), (8, 8, 128, 1, 1, 1 << 40))


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would run, on addresses of nothing")
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_paged_attention_takes_wide_calls(lib, cache):
    """Calls below the documented limit get as far as the launch, which fails here."""
    for hq, hkv, d, T, S, positions in WIDE_CALLS:
        cfg = _cfg(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=1024, cache_dtype=cache)
        kv = _kv(num_seqs=S, block_table_stride=min(positions // 1024, 2 ** 31 - 1),
                 page_stride=1 << 20)
        assert _attn(lib, cfg=cfg, T=T, kv=kv, qs=hq * d) == binding.ERR_CUDA, (hq, d, T)


UNITS = r"""
#include <cstdio>
#include "attn_plan.h"
using namespace gbmoe;
int main() {
  int G, hkv, D, fp8, T, S;
  double cap;
  while (scanf("%d %d %d %d %d %d %lf", &G, &hkv, &D, &fp8, &T, &S, &cap) == 7) {
    const int shift = unit_shift(G, hkv, D, fp8 != 0, T, S, cap);
    printf("%d %d %d\n", shift, tile_cost(shift, D), unit_cost(shift, D, fp8 != 0, true));
  }
  return 0;
}
"""


def test_units_fit_and_the_documented_limit_holds(tmp_path):
    """No line of a chosen launch leaves 32 bits at any lengths, and what the header says is enough
    is enough, on either side of each limit."""
    (tmp_path / "units.cpp").write_text(UNITS)
    subprocess.run(["g++", "-std=c++17", "-I", build_mod.CSRC, str(tmp_path / "units.cpp"), "-o",
                    str(tmp_path / "units")], check=True)
    rng = random.Random(11)
    cases = [(hq // hkv, hkv, d, fp8, T, S, P) for hq, hkv, d, T, S, P in WIDE_CALLS
             for fp8 in (0, 1)]
    for _ in range(4000):
        hkv = rng.choice([1, 2, 8, 64, 1024])
        G = rng.choice([1, 2, 4, 8, 7, 1024 // hkv])
        G = max(1, min(G, 1024 // hkv))
        S = min(8192, int(2 ** rng.uniform(0, 13.01)))
        T = min(1 << 22, (1 << 30) // (G * hkv), max(1, int(S * 2 ** rng.uniform(-2, 12))))
        rows = T * G / S
        # at a limit, or anywhere
        units = hkv * (T * G / rng.choice([8, 256]) + S)
        P = max(1, 128 * (2 ** 31 / units / rng.choice([1, 5]) + rng.choice([-5, -4, -3.9, -5.1])))
        if rng.random() < 0.3 or rows > 1e6:
            P = 2 ** rng.uniform(0, 34)
        cases.append((G, hkv, rng.choice([64, 128]), rng.randint(0, 1), T, S, P))
    out = subprocess.run([str(tmp_path / "units")], text=True, capture_output=True, check=True,
                         input="\n".join(" ".join(map(str, c)) for c in cases)).stdout.split("\n")
    taken, refused = set(), 0
    for (G, hkv, d, fp8, T, S, P), line in zip(cases, out):
        shift, tile, extra = (int(x) for x in line.split())
        P = min(P, 2 ** 30)
        few = hkv * (T * G / 8 + S) * (P / 128 + 5)
        many = hkv * (T * G / 256 + S) * (P / 128 + 5) * (5 if d == 64 else 1)
        enough = few < 2 ** 31 or (T * G > 16 * S and many < 2 ** 31)
        assert shift in (3, 4, 8) if enough else shift in (0, 3, 4, 8)
        refused += shift == 0
        if not shift:
            continue
        taken.add((shift, T * G > 16 * S, d))
        # rows spread to make the most units: one more than they fill for every sequence
        units = hkv * (T * G // 2 ** shift + S)
        assert units * (-(-int(P) // 128) * tile + extra) < 2 ** 31 - 8
        if T * G <= 8 * S:
            assert shift == 3
    assert refused > 100 and {(8, True, 64), (8, True, 128), (3, True, 64), (4, False, 128)} <= taken
    assert all(int(l.split()[0]) for l in out[:2 * len(WIDE_CALLS)])


def test_cache_scales_have_a_finite_reciprocal(lib):
    """1e-39 is a finite scale whose reciprocal is not: zeros would become NaN codes."""
    for name in ("k_scale", "v_scale"):
        cfg = _cfg(cache_dtype="fp8", **{name: 1e-39})
        assert _append(lib, cfg=cfg) == BAD and _attn(lib, cfg=cfg) == BAD
        assert lib.moe_paged_attention_workspace_size(ctypes.byref(cfg)) == 0
        cfg = _cfg(cache_dtype="fp8", **{name: 3e-39})
        assert lib.moe_paged_attention_workspace_size(ctypes.byref(cfg)) > 0


# rows per unit (log2), cost of a tile in units of half the rows and in the others, cost of a unit
LAUNCHED = [(3, 1, 1, e) for e in (0, 1, 2, 3)] + [(4, 1, 1, 4), (4, 1, 1, 6), (8, 1, 1, 3),
                                                   (8, 4, 5, 15)]


def test_cut_units_join_in_the_launched_shapes(tmp_path):
    """The costs that the kernels are launched with: every tile of a unit is computed once, in
    order, and what joins a cut unit's pieces finds them all. Where a tile costs 1 they are in
    neighbouring CTAs; else a CTA between two pieces may have none. Among the cases: ranges within
    one unit's extra cost."""
    (tmp_path / "plan.cpp").write_text(PLAN)
    subprocess.run(["g++", "-std=c++17", "-I", build_mod.CSRC, str(tmp_path / "plan.cpp"), "-o",
                    str(tmp_path / "plan")], check=True)
    (tmp_path / "units.cpp").write_text(UNITS)
    subprocess.run(["g++", "-std=c++17", "-I", build_mod.CSRC, str(tmp_path / "units.cpp"), "-o",
                    str(tmp_path / "units")], check=True)
    rng = random.Random(19)
    cases = []
    for shape in LAUNCHED:
        for _ in range(150):
            S = rng.choice([1, 1, 2, 5, 12, 40])
            seqs = []
            for _ in range(S):
                n = rng.choice([0, 1, 1, 1, 2, 4, 17, 130])
                seqs.append((n, max(0, rng.choice([n, n + 1, n - 2, n + 128, n + 700, n + 9000]))))
            if not any(n for n, _ in seqs):
                seqs[0] = (1, 3)
            cases.append((shape, rng.choice([1, 2, 4, 7, 16]), rng.choice([1, 2, 8]),
                          int(rng.random() < 0.8), rng.choice([0, 0, 1, 129, 1000]),
                          rng.choice([2, 148, 152, 152, 152]), seqs))
    for _ in range(300):       # units of one half and of two after each other: tiles of 4 and of 5
        seqs = [(n, n + 128 * rng.randint(0, 40)) for n in rng.choices([100, 200], k=4)]
        cases.append((LAUNCHED[-1], 1, 1, 0, 0, 152, seqs))
    text = "\n".join(f"{G} {hkv} {sh} {extra} {half} {full} {causal} {window} {g} {len(seqs)} "
                     + " ".join(f"{n} {L}" for n, L in seqs)
                     for (sh, half, full, extra), G, hkv, causal, window, g, seqs in cases)
    out = subprocess.run([str(tmp_path / "plan")], input=text, text=True, capture_output=True,
                         check=True).stdout.splitlines()
    assert len(out) == len(cases)
    cut, skipped, idle = 0, 0, 0
    for (shape, G, hkv, causal, window, g, seqs), line in zip(cases, out):
        sh, half, full, extra = shape
        v = [int(x) for x in line.split()]
        pieces = [tuple(v[i:i + 8]) for i in range(0, len(v), 8)]   # c s head rb ta tb t0 tiles
        units, of = {}, {}
        for c, s, head, rb, ta, tb, t0, tiles in pieces:
            units.setdefault((s, head, rb), []).append((c, ta, tb, tiles))
            of.setdefault(c, []).append(((s, head, rb), ta > 0, tb < tiles))
        want = {(s, h, rb) for s, (n, _) in enumerate(seqs) for h in range(hkv)
                for rb in range(-(-n * G // 2 ** sh))}
        assert set(units) == want
        idle += max(of) + 1 - len(of)
        for u, ps in units.items():
            assert ps[0][1] == 0 and ps[-1][2] == ps[-1][3]
            assert all(a[2] == b[1] and a[0] < b[0] for a, b in zip(ps, ps[1:]))
            held = [p[0] for p in ps]
            gaps = held != list(range(held[0], held[-1] + 1))
            assert not (gaps and full == 1)
            cut += len(ps) > 1
            skipped += gaps
        for c, ps in of.items():
            # at most the first piece is of a unit begun before, and the last of one left behind
            assert not any(p[1] for p in ps[1:]) and not any(p[2] for p in ps[:-1])
            u, mid, leaves = ps[-1]
            if not leaves or mid:
                continue
            # the joining kernel's rule: up to the first later CTA whose first piece ends a unit
            # that was begun before it, whatever lies between with such a piece
            rest, found = [], [c]
            for d in sorted(x for x in of if x > c):
                if of[d][0][1]:
                    found.append(d)
                    rest.append(of[d][0][0])
                    if not of[d][0][2]:
                        break
            assert found == [p[0] for p in units[u]] and all(x == u for x in rest)
    assert cut > 1000 and skipped > 0 and idle > 100
    # these are the costs that the launches take
    ask = [(1, 1, d, fp8, T, 16, 100.0) for d in (64, 128) for fp8 in (0, 1) for T in (16, 256, 4096)]
    lines = subprocess.run([str(tmp_path / "units")], text=True, capture_output=True, check=True,
                           input="\n".join(" ".join(map(str, a)) for a in ask)).stdout.splitlines()
    shapes = {(sh, full, extra) for sh, _, full, extra in LAUNCHED}
    assert {tuple(int(x) for x in line.split()) for line in lines} <= shapes
