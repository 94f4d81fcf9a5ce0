// Paged attention of few query rows per kv head (single tokens, short drafts): units of 16 rows
// (token, query head of the group), bound by reading K and V once from HBM.
//
// One persistent CTA per SM takes an equal share of all sequences' key tiles (attn_plan.h). Warp
// 8 streams tiles of 128 keys through a ring of shared-memory stages with TMA, one box per page
// and 128 bytes of the head, 128-byte swizzled; the page ids of a tile are fetched one tile
// ahead. Warps 0..7 own 16 keys of every tile each:
//   S = Q K^T (16 x 16 by mma.m16n8k16, fp32), p = 2^(S - m), O += P V,
// with a running maximum, sum and O of their own, so that no tile needs a barrier between
// warps; they are joined through shared memory at the end of a piece. A 16-row product leaves
// the tensor cores almost idle whatever form it takes, and this one needs neither tensor
// memory nor a trip of P through shared memory.
//
// bf16 cache: bf16 products, P rounded to bf16. e4m3 cache: codes become f16 (exact) and the
// products run in f16 with Q rounded (saturating) and P rounded to f16; the scales of k and v
// are applied to the scores and to the output.
#include <cuda_fp16.h>

#include "attn.cuh"

namespace gbmoe {
namespace {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * (kDecWarps + 1);
constexpr int kDecBR = 16;
constexpr uint32_t kDecRing = 160 * 1024;
constexpr uint32_t kDecJoin = 64 * 1024;  // 8 warps x 16 rows x 128 columns fp32
constexpr size_t kDecSmem = 1024 + kDecRing + kDecJoin + 2048;
static_assert(kDecSmem <= 232448, "shared memory per CTA exceeded");

template <bool FP8, int D>
struct Dec {
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kPitch = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a box row
  static constexpr int kParts = kRowBytes / kPitch;                 // boxes across a row
  static constexpr uint32_t kStage = kAttnTK * kRowBytes;           // one K or V tile
  static constexpr int kStages = kDecRing / kStage < 10 ? kDecRing / kStage : 10;
  static constexpr uint32_t kSwz = kPitch == 128 ? 0x70u : 0x30u;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, "
        "%7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
// Two e4m3 bytes (low byte first) as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
// Barrier of the consumer warps; whether any of them came with `failed` (the same answer for all,
// so that they leave together).
__device__ __forceinline__ bool consumers_sync(bool failed) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)failed), "n"(32 * kDecWarps)
      : "memory");
  return any != 0;
}
// Spin (bounded) until a copy in flight has landed, so that the CTA does not exit under it.
__device__ __noinline__ void land(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 10000000ull) return;
}

struct DecMaps {
  CUtensorMap k, v;
};

template <bool FP8, int D>
__global__ void __launch_bounds__(kDecThreads, 1)
    attn_decode_kernel(const __grid_constant__ DecMaps maps, const __grid_constant__ AttnArgs a,
                       const __grid_constant__ AttnShape sh) {
  using T = Dec<FP8, D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw0);
  float* join = reinterpret_cast<float*>(smem + kDecRing);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kDecRing + kDecJoin);
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (10 + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 20);
  float2* wml = reinterpret_cast<float2*>(bars + 24);              // [16 rows][8 warps] = 1 KB
  long long* wsum = reinterpret_cast<long long*>(bars + 24 + 128);  // 32
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kDecWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch(&maps.k);
    tma_prefetch(&maps.v);
  }
  // the line of tiles is laid out in the ring before the first copy lands there
  AttnCursor cur = attn_plan(a.b, sh, reinterpret_cast<long long*>(smem), wsum);
  fence_async_proxy();
  __syncthreads();
  int* status = a.b.status;

  if (warp == kDecWarps) {
    // ------------------------------------------------------------ tile copies
    const int ps = 1 << a.b.page_shift;
    const int box_rows = min(ps, kAttnTK);
    const int boxes = kAttnTK / box_rows * T::kParts;  // <= 32: pages of at least 8 rows
    const int pl = lane / T::kParts, part = lane % T::kParts;
    const uint32_t box_bytes = (uint32_t)box_rows * T::kPitch;
    uint32_t slot = 0, phase = 0, issued = 0;
    bool ok = true;
    while (ok && cur.left > 0) {
      AttnPiece p;
      if (!next_piece(a.b, sh, cur, p)) break;
      // this lane's box of tile t: whether it holds any key of the unit, and its page
      auto live_at = [&](int t) {
        const int j = (p.u.t0 + t) * kAttnTK + pl * box_rows;
        return lane < boxes && j < p.u.hi && j + box_rows > p.u.lo;
      };
      auto page_at = [&](int t) {
        return t < p.tb && live_at(t)
                   ? page_of(a.b, p.s, (p.u.t0 + t) * kAttnTK + pl * box_rows)
                   : 0;
      };
      int page = page_at(p.ta);
      for (int t = p.ta; ok && t < p.tb; ++t) {
        const int next = page_at(t + 1);
        const bool live = live_at(t);
        const uint32_t bytes = box_bytes * __popc(__ballot_sync(0xffffffffu, live));
        const int y = ((p.u.t0 + t) * kAttnTK + pl * box_rows) & (ps - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (!wait_fast(empty(slot), phase ^ 1u, abort_flag, status)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_expect_tx(full(slot), bytes);
          __syncwarp();
          if (live)
            tma_load_4d(base + slot * T::kStage + (uint32_t)part * kAttnTK * T::kPitch +
                            (uint32_t)pl * box_bytes,
                        kv ? &maps.v : &maps.k, full(slot), part * (FP8 ? T::kPitch : 64), y,
                        p.head, page);
          ++issued;
          if (++slot == T::kStages) {
            slot = 0;
            phase ^= 1u;
          }
        }
        page = next;
      }
    }
    if (*abort_flag && lane == 0)  // let what is in flight land before the CTA can exit
      for (uint32_t j = issued > (uint32_t)T::kStages ? issued - T::kStages : 0; j < issued; ++j)
        land(full(j % T::kStages), (j / T::kStages) & 1u);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ 16 keys of every tile
    const AttnScratch sc = attn_scratch(a.scratch, kDecBR);
    AttnRec rec;
    rec.starts = rec.mid = rec.ends = rec.s = rec.head = rec.rb = 0;
    const int g = lane >> 2, c = lane & 3;
    uint32_t slot = 0, phase = 0;
    bool ok = true;
    auto next_stage = [&]() {
      if (++slot == T::kStages) {
        slot = 0;
        phase ^= 1u;
      }
    };
    auto swz = [](uint32_t off) { return off ^ ((off >> 3) & T::kSwz); };
    while (cur.left > 0) {
      AttnPiece p;
      if (!next_piece(a.b, sh, cur, p)) break;
      const int rows = min(kDecBR, p.q.n * sh.G - p.rb * kDecBR);
      // this lane's two rows: their query vectors as mma fragments, and their keys
      uint32_t qf[D / 16][4];
      KeyRange kr[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = g + 8 * h;
        const bool valid = r < rows;
        const int rr = p.rb * kDecBR + (valid ? r : 0);
        const int i = rr / sh.G;
        kr[h] = key_range(p.q, i, sh.causal, sh.window);
        if (!valid) kr[h].hi = kr[h].lo = 0;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                   (size_t)(p.q.q0 + i) * a.q_stride +
                                   (size_t)(p.head * sh.G + rr % sh.G) * D;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t lo = 0u, hi = 0u;
          if (valid && FP8) {
            // e4m3 fragments hold columns 4c .. 4c + 3 of each 16: Q's follow that order
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + 16 * k + 4 * c));
            const float2 x = unpack_bf16x2(w.x), y = unpack_bf16x2(w.y);
            auto cut = [](float v) { return v > 65504.f ? 65504.f : (v < -65504.f ? -65504.f : v); };
            lo = pack_f16x2(cut(x.x), cut(x.y));
            hi = pack_f16x2(cut(y.x), cut(y.y));
          } else if (valid) {
            lo = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * c));
            hi = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * c));
          }
          qf[k][h] = lo;
          qf[k][2 + h] = hi;
        }
      }
      // keys that every row of the unit attends need no mask
      const KeyRange k0 = key_range(p.q, p.u.i0, sh.causal, sh.window);
      const KeyRange k1 = key_range(p.q, p.u.i1, sh.causal, sh.window);
      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

      for (int t = p.ta; t < p.tb; ++t) {
        const int j0 = (p.u.t0 + t) * kAttnTK + warp * 16;  // this warp's keys
        const bool some = j0 < p.u.hi && j0 + 16 > p.u.lo;
        uint32_t pf[4];
        if (!wait_fast(full(slot), phase, abort_flag, status)) {
          ok = false;
          break;
        }
        if (some) {
          const uint32_t st = base + slot * T::kStage;
          float s[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
          if (FP8) {
            // one ldmatrix: keys 0-7 and 8-15 x 32 columns, 16 bytes per 8x8 matrix row
            const uint32_t row = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              uint32_t w[4];
              ldsm4(st + swz(row * T::kPitch + k * 32 + ((lane >> 3) & 1) * 16), w);
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  mma16816<true>(s[n], qf[2 * k + h], e4m3x2_f16(w[2 * n + h]),
                                 e4m3x2_f16(w[2 * n + h] >> 16));
            }
          } else {
            const uint32_t row = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              uint32_t w[4];
              const uint32_t col = (k % 4) * 32 + ((lane >> 3) & 1) * 16;
              ldsm4(st + (k / 4) * (kAttnTK * 128) + swz(row * 128 + col), w);
              mma16816<false>(s[0], qf[k], w[0], w[1]);
              mma16816<false>(s[1], qf[k], w[2], w[3]);
            }
          }
          // scores in log2 units; keys that a row does not attend drop out
          const bool mask = j0 < max(k0.lo, k1.lo) || j0 + 16 > min(k0.hi, k1.hi);
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v = s[n][e] * a.scale_log2;
              if (mask) {
                const int j = j0 + 8 * n + 2 * c + (e & 1);
                if (j < kr[e >> 1].lo || j >= kr[e >> 1].hi) v = -INFINITY;
              }
              s[n][e] = v;
            }
          float mn[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            mn[h] = fmaxf(m[h], x);
          }
          if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float f = mn[h] > m[h] ? ex2(m[h] - mn[h]) : 1.f;
              m[h] = mn[h];
              l[h] *= f;
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                o[i][2 * h] *= f;
                o[i][2 * h + 1] *= f;
              }
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mm = m[h] == -INFINITY ? 0.f : m[h];
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = ex2(s[i >> 1][2 * h + (i & 1)] - mm);
            l[h] += (e[0] + e[1]) + (e[2] + e[3]);
            pf[h] = pack16<FP8>(e[0], e[1]);
            pf[2 + h] = pack16<FP8>(e[2], e[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(slot));
        next_stage();
        if (!wait_fast(full(slot), phase, abort_flag, status)) {
          ok = false;
          break;
        }
        if (some) {
          const uint32_t st = base + slot * T::kStage;
          if (j0 < p.u.lo || j0 + 16 > p.u.hi) {
            // v of positions that no row attends: 0, whatever the page holds (0 * NaN = NaN)
            for (int i = lane; i < 16 * (T::kRowBytes / 16); i += 32) {
              const int r = i / (T::kRowBytes / 16), x = i % (T::kRowBytes / 16);
              if (j0 + r < p.u.lo || j0 + r >= p.u.hi)
                sts128(st + (x * 16 / T::kPitch) * (kAttnTK * T::kPitch) +
                           (warp * 16 + r) * T::kPitch + x * 16 % T::kPitch,
                       make_uint4(0u, 0u, 0u, 0u));
            }
            __syncwarp();
            fence_async_proxy();  // before the stage's next copy
          }
          const uint32_t row = warp * 16 + (lane & 15);
          if (FP8) {
            // transposed 8x8 matrices of byte pairs: columns 2n and 2n + 1 of two keys a word
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              uint32_t w[4];
              ldsm4t(st + swz(row * T::kPitch + k * 32 + (lane >> 4) * 16), w);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t sel = e ? 0x0031u : 0x0020u;
                  mma16816<true>(o[4 * k + 2 * h + e], pf,
                                 e4m3x2_f16(__byte_perm(w[2 * h], 0u, sel)),
                                 e4m3x2_f16(__byte_perm(w[2 * h + 1], 0u, sel)));
                }
            }
          } else {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              uint32_t w[4];
              const uint32_t col = (k % 4) * 32 + (lane >> 4) * 16;
              ldsm4t(st + (k / 4) * (kAttnTK * 128) + swz(row * 128 + col), w);
              mma16816<false>(o[2 * k], pf, w[0], w[1]);
              mma16816<false>(o[2 * k + 1], pf, w[2], w[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(slot));
        next_stage();
      }

      // ---------------------------------------------------------- the piece's result
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int r = g + 8 * h;
        if (c == 0) wml[r * kDecWarps + warp] = make_float2(m[h], l[h]);
        if (r < rows) {
          float* dst = join + (warp * kDecBR + r) * D;
          if (FP8) {
            // fragments (h2, e): columns 32 k + 16 h2 + 4 c + e and + 2
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              *reinterpret_cast<float4*>(dst + 16 * k + 4 * c) =
                  make_float4(o[2 * k][2 * h], o[2 * k + 1][2 * h], o[2 * k][2 * h + 1],
                              o[2 * k + 1][2 * h + 1]);
          } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<float2*>(dst + 8 * i + 2 * c) =
                  make_float2(o[i][2 * h], o[i][2 * h + 1]);
          }
        }
      }
      if (consumers_sync(!ok)) break;
      const int slot_out = p.first() ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
      for (int i = threadIdx.x; i < rows * (D / 4); i += 32 * kDecWarps) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float2 ml[kDecWarps];
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          ml[w] = wml[r * kDecWarps + w];
          M = fmaxf(M, ml[w].x);
        }
        const float Ms = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float f = ex2(ml[w].x - Ms);
          const float4 x = *reinterpret_cast<const float4*>(join + (w * kDecBR + r) * D + d);
          L = fmaf(f, ml[w].y, L);
          v.x = fmaf(f, x.x, v.x);
          v.y = fmaf(f, x.y, v.y);
          v.z = fmaf(f, x.z, v.z);
          v.w = fmaf(f, x.w, v.w);
        }
        if (p.whole()) {
          const int rr = p.rb * kDecBR + r;
          const size_t orow = (size_t)(p.q.q0 + rr / sh.G) * a.hq + p.head * sh.G + rr % sh.G;
          const float inv = L == 0.f ? 0.f : a.v_scale / L;
          uint2 w;
          w.x = pack_bf16x2(v.x * inv, v.y * inv);
          w.y = pack_bf16x2(v.z * inv, v.w * inv);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + d) = w;
          if (a.lse && d == 0)
            a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        } else {
          const size_t at = (size_t)slot_out * kDecBR + r;
          *reinterpret_cast<float4*>(sc.o + at * D + d) = v;
          if (d == 0) sc.ml[at] = make_float2(M, L);
        }
      }
      if (p.first() && !p.last()) {
        rec.starts = 1;
        rec.s = p.s;
        rec.head = p.head;
        rec.rb = p.rb;
      } else if (!p.first()) {
        rec.mid = 1;
        rec.ends = p.last();
      }
      consumers_sync(false);  // the join area is free again
    }
    if (threadIdx.x == 0) sc.rec[blockIdx.x] = rec;
  }
  __syncthreads();
}

template <bool FP8, int D>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t stream) {
  static int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    const cudaError_t e = cudaFuncSetAttribute(
        attn_decode_kernel<FP8, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDecSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  DecMaps maps;
  if (!make_cache_map(&maps.k, a.c.k, a) || !make_cache_map(&maps.v, a.c.v, a))
    return cudaErrorInvalidValue;
  AttnShape sh;
  sh.G = a.hq / a.hkv;
  sh.hkv = a.hkv;
  sh.br_shift = 4;
  static_assert(kDecBR == 1 << 4, "rows per unit");
  sh.extra = 0;
  sh.causal = a.causal;
  sh.window = a.window;
  const int ctas = num_sms() < kAttnMaxCtas ? num_sms() : kAttnMaxCtas;
  const cudaError_t e = launch_kernel(attn_decode_kernel<FP8, D>, dim3(ctas), dim3(kDecThreads),
                                      kDecSmem, stream, maps, a, sh);
  if (e != cudaSuccess) return e;
  return launch_attn_join(a, sh, ctas, stream);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t stream) {
  if (a.fp8)
    return a.D == 64 ? launch_typed<true, 64>(a, stream) : launch_typed<true, 128>(a, stream);
  return a.D == 64 ? launch_typed<false, 64>(a, stream) : launch_typed<false, 128>(a, stream);
}

}  // namespace gbmoe
