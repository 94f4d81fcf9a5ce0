"""Inputs and 64-bit references of the decoder-block operator tests (CPU arithmetic)."""
import math

import torch

BF16, FP8_HALF, FP32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24   # half a step, relative
E4M3_SUB = 2.0 ** -10                                     # half a step of e4m3's subnormals


def norm_reference(x, residual, weight, eps):
    h = x.double() + (0 if residual is None else residual.double())
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * weight.double()


class Paged:
    """Sequences (new tokens, total positions) over a paged cache on the CPU, with a block table
    in random page order; what no sequence owns is NaN, entries past a sequence's end are wild."""

    def __init__(self, seqs, hkv, d, page, cache="bf16", seed=0, spare=2, std=1.0, k_scale=1.0,
                 v_scale=1.0, wild=2 ** 31 - 1):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.page, self.cache, self.hkv, self.d = seqs, page, cache, hkv, d
        self.k_scale, self.v_scale = k_scale, v_scale
        need = [-(-L // page) for _, L in seqs]
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g)
        self.table = torch.full((len(seqs), max(max(need), 1) + 1), wild, dtype=torch.int32)
        at = 0
        self.rows = []                          # flat cache rows of each sequence's positions
        for s, n in enumerate(need):
            ids = order[at:at + n]
            at += n
            self.table[s, :n] = ids.int()
            L = seqs[s][1]
            self.rows.append((ids[:, None] * page + torch.arange(page)).reshape(-1)[:L])
        self.cu = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).int()
        self.kv_lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
        self.T = int(self.cu[-1])
        flat = (self.num_pages * page, hkv, d)
        self.k, self.v = (self._poisoned(flat) for _ in range(2))
        for r in self.rows:
            for c, sc in ((self.k, k_scale), (self.v, v_scale)):
                x = torch.randn(len(r), hkv, d, generator=g) * std / sc
                self.put(c, r, x)
        self.gen = g

    def _poisoned(self, flat):
        if self.cache == "fp8":
            return torch.full(flat, 0x7F, dtype=torch.uint8)
        return torch.full(flat, math.nan, dtype=torch.bfloat16)

    def put(self, cache, rows, x):
        if self.cache == "fp8":
            cache[rows] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            cache[rows] = x.to(torch.bfloat16)

    def shaped(self, cache):
        return cache.view(self.num_pages, self.page, self.hkv, self.d)

    def values(self, cache, scale):
        if self.cache == "fp8":
            return cache.view(torch.float8_e4m3fn).double() * scale
        return cache.double()


def attention_reference(p: Paged, q, causal=True, window=0, scale=None):
    """(out, lse, bound, lse_bound) in 64 bits: per element, the error that the roundings of the
    kernel allow: the output's rounding, the weights' rounding to 16 bits, fp32 scores (a sum of
    d products) and fp32 sums over the keys."""
    T, hq, d = q.shape
    G = hq // p.hkv
    scale = d ** -0.5 if scale is None else scale
    out, bound = (torch.zeros(T, hq, d, dtype=torch.float64) for _ in range(2))
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    lse_bound = torch.zeros(T, hq, dtype=torch.float64)
    for s, (n, L) in enumerate(p.seqs):
        k = p.values(p.k, p.k_scale)[p.rows[s]]
        v = p.values(p.v, p.v_scale)[p.rows[s]]
        t0 = int(p.cu[s])
        pos = L - n + torch.arange(n)[:, None]
        j = torch.arange(L)[None]
        seen = torch.ones(n, L, dtype=torch.bool)
        if causal:
            seen &= j <= pos
        if window:
            seen &= j > pos - window
        for h in range(hq):
            qh, kh, vh = q[t0:t0 + n, h].double(), k[:, h // G], v[:, h // G]
            z = (qh @ kh.T * scale).masked_fill(~seen, -math.inf)
            some = seen.any(1)
            m = torch.where(some, z.amax(1) if L else torch.zeros(n).double(), 0.0)
            e = torch.exp(z - m[:, None])
            tot = e.sum(1)
            w = e / torch.where(some, tot, 1.0)[:, None]
            o = w @ vh
            size = (qh.abs() @ kh.abs().T * scale).masked_fill(~seen, 0.0)
            es = (d + 8) * FP32 * (size.amax(1) if L else torch.zeros(n).double()) + 8 * FP32
            a = w @ vh.abs()
            keys = seen.sum(1).double()
            out[t0:t0 + n, h] = o
            vmax = vh.abs().max() if L else 0.0
            bound[t0:t0 + n, h] = (BF16 * o.abs() + a * (BF16 + 2 * es + 2 * keys * FP32)[:, None]
                                   + (keys * FP32 * vmax / torch.where(some, tot, 1.0))[:, None])
            lse[t0:t0 + n, h] = torch.where(some, m + tot.log(), -math.inf)
            lse_bound[t0:t0 + n, h] = es + keys * FP32 + 4 * FP32 * (m.abs() + tot.log().abs()
                                                                     .nan_to_num(0, 0, 0))
    return out, lse, bound, lse_bound


def rotate_reference(x, cos, sin, interleaved):
    """(rotated, sum of the products' magnitudes) of x [n, heads, d] in 64 bits."""
    R = 2 * cos.shape[-1]
    y, size = x.double().clone(), x.double().abs()
    a = slice(0, R, 2) if interleaved else slice(0, R // 2)
    b = slice(1, R, 2) if interleaved else slice(R // 2, R)
    c, s = cos.double()[:, None], sin.double()[:, None]
    xa, xb = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    size[..., a] = (xa * c).abs() + (xb * s).abs()
    size[..., b] = (xb * c).abs() + (xa * s).abs()
    return y, size
