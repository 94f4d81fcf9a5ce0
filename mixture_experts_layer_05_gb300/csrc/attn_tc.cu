// Paged attention of many query rows per kv head (prompts, chunks of new tokens, and the single
// tokens that ride along): units of 256 rows (token, query head of the group) on the 5th
// generation tensor cores.
//
// One persistent CTA per SM takes an equal share of all units' key tiles (attn_plan.h). The 256
// rows are two halves of 128, each with its own softmax warpgroup, so that the tensor core works
// for one half while the other's softmax runs. Per tile of 128 keys and half:
//   S = Q K^T    tcgen05.mma, Q and K in shared memory, 128 x 128 fp32 in tensor memory
//   p = 2^(s - m)  one thread per row: the row's maximum, sum and exponentials in registers; P
//                goes back to tensor memory as 16-bit pairs over S's own columns
//   O += P V     tcgen05.mma with A = P in tensor memory and V as it lies in the pages (keys
//                down, columns across: the MN-major operand form), 128 x D fp32
// m is kept until a row's maximum has grown by more than 2^8 (the weights stay below 256, and
// their sum in fp32 loses nothing): O is rescaled in tensor memory only then.
//
//   warps 0-3, 4-7   softmax of half 0 / 1; they also bring the unit's Q into shared memory (the
//                    next piece's while the last product runs) and write the piece's result
//   warp 8           MMA issue (one thread)
//   warp 9           tile copies: TMA, one box per page and 128 bytes of the head; page ids one
//                    tile ahead
//   warps 10, 11     e4m3 cache only: codes to f16 (exact) into the operand tiles
//
// Tensor memory: S/P of half h at columns 128 h, O of half h at 256 + 128 h. Operand order in
// the ring: K0, K1, V0, K2, V1, ..., so that the next scores are under way before a tile's
// weights are. bf16 cache: bf16 products; e4m3: f16 products with Q rounded to f16 (saturating).
#include <cuda_fp16.h>

#include "attn.cuh"

namespace gbmoe {
namespace {

constexpr int kTcBR = 256;
constexpr int kTcMmaWarp = 8, kTcCopyWarp = 9, kTcCvtWarp = 10;
constexpr int kTcCvtWarps = 2;
constexpr float kTcSlack = 8.f;  // log2 growth of a row's maximum that O tolerates

template <bool FP8, int D>
struct Tc {
  static constexpr int kThreads = FP8 ? 32 * (kTcCvtWarp + kTcCvtWarps) : 32 * kTcCvtWarp;
  static constexpr uint32_t kTile = kAttnTK * D * 2;        // one operand tile (16 bit)
  static constexpr uint32_t kRawTile = kAttnTK * D;         // one tile of codes
  static constexpr int kRaw = FP8 ? 4 : 0;                  // code stages
  static constexpr int kStages = FP8 ? 3 : 5;               // operand stages
  static constexpr uint32_t kQ = 2 * kTile;
  static constexpr uint32_t kRawPitch = D < 128 ? D : 128;  // bytes of a code row
  static constexpr uint32_t kRawSwz = kRawPitch == 128 ? 0x70u : 0x30u;
  static constexpr size_t kSmem = 1024 + kQ + kStages * kTile + kRaw * kRawTile + 1024;
  static_assert(kSmem <= 232448, "shared memory per CTA exceeded");
  static_assert((kAttnMaxSeqs + 1) * 8 <= kQ + kStages * kTile, "the plan lies in Q and the ring");
};

// Instruction descriptor of kind::f16 (format 1 bf16, 0 f16), fp32 D, M = 128, A K-major; B
// K-major or (vt) MN-major.
__host__ __device__ constexpr uint32_t idesc_attn(bool f16, int N, bool vt) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (vt ? 1u << 16 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// V tile: MN-major, 128-byte swizzle: rows of 64 columns, 8-key groups 1024 bytes apart, the two
// 64-column halves one half tile apart.
__device__ __forceinline__ uint64_t sdesc_v(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((kAttnTK * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
      "%27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Four e4m3 bytes as two f16 pairs (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
}
// Two bf16 as an f16 pair, saturating (NaN stays NaN).
__device__ __forceinline__ uint32_t bf16x2_f16(uint32_t w) {
  const float2 f = unpack_bf16x2(w);
  auto cut = [](float v) { return v > 65504.f ? 65504.f : (v < -65504.f ? -65504.f : v); };
  return pack_f16x2(cut(f.x), cut(f.y));
}
// Spin (bounded) until a copy in flight has landed, so that the CTA does not exit under it.
__device__ __noinline__ void land(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 10000000ull) return;
}

struct TcMaps {
  CUtensorMap k, v;
};

// A ring position.
struct Ring {
  uint32_t slot, phase;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

template <bool FP8, int D>
__global__ void __launch_bounds__(Tc<FP8, D>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ AttnArgs a,
                   const __grid_constant__ AttnShape sh) {
  using T = Tc<FP8, D>;
  constexpr uint32_t kHalf = kAttnTK * 128;  // a 64-column half of an operand tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw0);
  const uint32_t q_base = base, ring = base + T::kQ, codes = ring + T::kStages * T::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::kQ + T::kStages * T::kTile +
                                               T::kRaw * T::kRawTile);
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };           // operand stage filled
  auto empty = [&](int s) { return bar0 + 8u * (5 + s); };    // ... and read by its MMAs
  auto q_full = [&](int g) { return bar0 + 8u * (10 + g); };
  auto s_full = [&](int g) { return bar0 + 8u * (12 + g); };
  auto p_full = [&](int g) { return bar0 + 8u * (14 + g); };
  auto pv_done = [&](int g) { return bar0 + 8u * (16 + g); };
  auto raw_full = [&](int s) { return bar0 + 8u * (18 + s); };
  auto raw_empty = [&](int s) { return bar0 + 8u * (22 + s); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 26);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  long long* wsum = reinterpret_cast<long long*>(bars + 28);  // 32
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = a.b.status;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(full(s), FP8 ? kTcCvtWarps : 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < T::kRaw; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), kTcCvtWarps);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(q_full(g), 4);
      mbar_init(s_full(g), 1);
      mbar_init(p_full(g), 4);
      mbar_init(pv_done(g), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch(&maps.k);
    tma_prefetch(&maps.v);
  }
  if (warp == kTcMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  AttnCursor cur = attn_plan(a.b, sh, reinterpret_cast<long long*>(smem), wsum);
  fence_async_proxy();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // a wait whose answer is the whole warp's (tcgen05 and warp barriers follow it)
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_fast(bar, parity, abort_flag, status)) != 0;
  };
  auto rows_of = [&](const AttnPiece& p) { return min(kTcBR, p.q.n * sh.G - p.rb * kTcBR); };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const AttnScratch sc = attn_scratch(a.scratch, kTcBR);
    const int g = warp >> 2;
    const int row = threadIdx.x & 127;                       // of this half
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128u * g, to = tmem + lanes + 256u + 128u * g;
    const uint32_t q_row = q_base + g * T::kTile + row * 128u;
    // the CTA's record in the workspace, by one thread
    auto note = [&](const AttnPiece& p) {
      if (threadIdx.x) return;
      AttnRec& rec = sc.rec[blockIdx.x];
      if (p.first() && !p.last()) {
        rec.s = p.s;
        rec.head = p.head;
        rec.rb = p.rb;
        rec.starts = 1;
      } else if (!p.first()) {
        rec.mid = 1;
        rec.ends = p.last();
      }
    };
    if (threadIdx.x == 0) sc.rec[blockIdx.x].starts = sc.rec[blockIdx.x].mid = sc.rec[blockIdx.x].ends = 0;
    // the next piece that has rows in this half
    auto fetch = [&](AttnPiece& p) {
      while (cur.left > 0) {
        p = next_piece(a.b, sh, cur);
        note(p);
        if (rows_of(p) > 128 * g) return true;
      }
      return false;
    };
    // A piece as this thread's row needs it.
    struct Job {
      int nt, j0;          // tiles, first key of the first
      int lo, hi;          // the row's keys
      int in_lo, in_hi;    // keys that every row of the unit attends
      int row;             // output row (token * heads + head), or the slot's; -1: no such row
      bool whole;
    } job;
    // Turns the piece into this thread's job and its query row into shared memory.
    auto begin = [&](const AttnPiece& p) {
      const int r = 128 * g + row, rr = p.rb * kTcBR + r;
      const bool valid = r < rows_of(p);
      const int tok = rr / sh.G, head = p.head * sh.G + rr % sh.G;
      const KeyRange k0 = key_range(p.q, p.u.i0, sh.causal, sh.window);
      const KeyRange k1 = key_range(p.q, p.u.i1, sh.causal, sh.window);
      const KeyRange kr = key_range(p.q, tok, sh.causal, sh.window);
      job.nt = p.tb - p.ta;
      job.j0 = (p.u.t0 + p.ta) * kAttnTK;
      job.lo = kr.lo;
      job.hi = valid ? kr.hi : 0;
      job.in_lo = max(k0.lo, k1.lo);
      job.in_hi = min(k0.hi, k1.hi);
      job.whole = p.whole();
      job.row = !valid ? -1
                : job.whole ? (p.q.q0 + tok) * a.hq + head
                            : (p.first() ? 2 * (int)blockIdx.x + 1 : 2 * (int)blockIdx.x) * kTcBR + r;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                 (size_t)(p.q.q0 + tok) * a.q_stride + (size_t)head * D;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (valid) v = __ldg(reinterpret_cast<const uint4*>(src) + c);
        if (FP8) {
          v.x = bf16x2_f16(v.x);
          v.y = bf16x2_f16(v.y);
          v.z = bf16x2_f16(v.z);
          v.w = bf16x2_f16(v.w);
        }
        sts128(q_row + (c / 8) * kHalf + (((c & 7) ^ (row & 7)) << 4), v);
      }
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(g));
    };
    bool have;
    {
      AttnPiece p;
      have = fetch(p);
      if (have) begin(p);
    }
    uint32_t tc = 0;  // tiles of this half so far
    while (have) {
      float m = -INFINITY, l = 0.f;   // m: the reference of the weights, raw score units
      bool ok = true;
      for (int t = 0; t < job.nt; ++t, ++tc) {
        if (!wait(s_full(g), tc & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_wait_ld(s[i]);
        const int j0 = job.j0 + t * kAttnTK;
        if (j0 < job.in_lo || j0 + kAttnTK > job.in_hi) {
          const int lo = job.lo - j0, hi = job.hi - j0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (32 * i + c < lo || 32 * i + c >= hi) s[i][c] = 0xff800000u;  // -inf
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
          for (int c = 1; c < 32; ++c) mx[i] = fmaxf(mx[i], __uint_as_float(s[i][c]));
        }
        const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        if (t == 0) {
          m = mn;
        } else if (__any_sync(0xffffffffu, mn > m && (mn - m) * a.scale_log2 > kTcSlack)) {
          // O catches up with the new maxima, once the product before this tile's is done
          if (!wait(pv_done(g), (tc - 1) & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f = mn > m ? ex2((m - mn) * a.scale_log2) : 1.f;
          m = mn;
          l *= f;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(to + 32 * i, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_st32(to + 32 * i, o);
          }
          tmem_wait_st();
        }
        const float off = m == -INFINITY ? 0.f : -m * a.scale_log2;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int k = 2 * c;
            const float e0 = ex2(fmaf(__uint_as_float(s[2 * h + k / 32][k % 32]), a.scale_log2, off));
            const float e1 =
                ex2(fmaf(__uint_as_float(s[2 * h + k / 32][k % 32 + 1]), a.scale_log2, off));
            sum[0] += e0;
            sum[1] += e1;
            w[c] = FP8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
          }
          tmem_st32(ts + 32 * h, w);
        }
        l += sum[0] + sum[1];
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(g));
      }
      if (!ok) break;
      // every score of the piece is out, so Q's place is free: the next piece's comes in while
      // the last product runs
      const Job done = job;
      {
        AttnPiece p;
        have = fetch(p);
        if (have) begin(p);
      }
      if (!wait(pv_done(g), (tc - 1) & 1u)) break;
      tc_fence_after();
      const float ml = m == -INFINITY ? -INFINITY : m * a.scale_log2;
      if (done.whole) {
        const float inv = l == 0.f ? 0.f : a.v_scale / l;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                              (size_t)done.row * D);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(to + 32 * i, o);
          tmem_wait_ld(o);
          if (done.row >= 0)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * k]) * inv,
                                   __uint_as_float(o[8 * c + 2 * k + 1]) * inv);
              dst[4 * i + c] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (a.lse && done.row >= 0)
          a.lse[done.row] = l == 0.f ? -INFINITY : (ml + log2f(l)) * 0.6931471805599453f;
      } else {
        uint4* dst = reinterpret_cast<uint4*>(sc.o + (size_t)done.row * D);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(to + 32 * i, o);
          tmem_wait_ld(o);
          if (done.row >= 0)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              dst[8 * i + c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
        if (done.row >= 0) sc.ml[done.row] = make_float2(ml, l);
      }
      tc_fence_before();
    }
  } else if (warp == kTcMmaWarp) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kIdS = idesc_attn(FP8, kAttnTK, false), kIdO = idesc_attn(FP8, D, true);
    Ring rg{0, 0};
    uint32_t qc[2] = {0, 0}, tcnt[2] = {0, 0};
    bool ok = true;
    auto take = [&](uint32_t& slot) {  // the next operand tile, filled
      if (!wait(full(rg.slot), rg.phase)) return false;
      slot = rg.slot;
      rg.next(T::kStages);
      return true;
    };
    auto scores = [&](int g, uint32_t slot) {
      if (lane == 0) {
        const uint64_t qa = sdesc_sw128(q_base + g * T::kTile);
        const uint64_t kb = sdesc_sw128(ring + slot * T::kTile);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = (k / 4) * kHalf + (k % 4) * 32;
          mma_bf16(tmem + 128u * g, sdesc_advance(qa, at), sdesc_advance(kb, at), kIdS, k > 0);
        }
        mma_commit(s_full(g));
      }
      __syncwarp();
    };
    while (ok && cur.left > 0) {
      const AttnPiece p = next_piece(a.b, sh, cur);
      const int halves = rows_of(p) > 128 ? 2 : 1;
      uint32_t ks = 0, vs = 0;
      if (!take(ks)) break;
      for (int g = 0; g < halves && ok; ++g) {
        ok = wait(q_full(g), qc[g]++ & 1u);
        tc_fence_after();
        if (ok) scores(g, ks);
      }
      if (!ok) break;
      if (lane == 0) mma_commit(empty(ks));
      for (int t = p.ta; ok && t < p.tb; ++t) {
        const bool more = t + 1 < p.tb;
        if ((more && !take(ks)) || !take(vs)) {
          ok = false;
          break;
        }
        const int j0 = (p.u.t0 + t) * kAttnTK;
        if (!FP8 && (j0 < p.u.lo || j0 + kAttnTK > p.u.hi)) {
          // v of positions that no row attends: 0, whatever the page holds (0 * NaN = NaN)
          const int lo = max(p.u.lo - j0, 0), hi = min(p.u.hi - j0, kAttnTK);
          for (int i = lane; i < kAttnTK * (D / 8); i += 32) {
            const int r = i / (D / 8), c = i % (D / 8);
            if (r < lo || r >= hi)
              sts128(ring + vs * T::kTile + (c / 8) * kHalf + r * 128 + (c & 7) * 16,
                     make_uint4(0u, 0u, 0u, 0u));
          }
          fence_async_proxy();
          __syncwarp();
        }
        for (int g = 0; g < halves; ++g) {
          if (!wait(p_full(g), tcnt[g]++ & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint64_t vb = sdesc_v(ring + vs * T::kTile);
#pragma unroll
            for (int k = 0; k < kAttnTK / 16; ++k)
              mma_ts(tmem + 256u + 128u * g, tmem + 128u * g + 8u * k,
                     sdesc_advance(vb, k * 2048), kIdO, t > p.ta || k > 0);
            mma_commit(pv_done(g));
          }
          __syncwarp();
          if (more) scores(g, ks);
        }
        if (ok && lane == 0) {
          mma_commit(empty(vs));
          if (more) mma_commit(empty(ks));
        }
        __syncwarp();
      }
    }
  } else if (warp == kTcCopyWarp) {
    // ------------------------------------------------------------ tile copies
    constexpr int kParts = FP8 ? 1 : D / 64;
    constexpr uint32_t kPitch = FP8 ? T::kRawPitch : 128;
    constexpr uint32_t kN = FP8 ? T::kRaw : T::kStages;
    const int ps = 1 << a.b.page_shift;
    const int box_rows = min(ps, kAttnTK);
    const int boxes = kAttnTK / box_rows * kParts;  // <= 32: pages of at least 8 rows
    const int pl = lane / kParts, part = lane % kParts;
    const uint32_t box_bytes = (uint32_t)box_rows * kPitch;
    Ring rg{0, 0};
    uint32_t issued = 0;
    bool ok = true;
    auto fullb = [&](uint32_t s) { return FP8 ? raw_full(s) : full(s); };
    auto emptyb = [&](uint32_t s) { return FP8 ? raw_empty(s) : empty(s); };
    while (ok && cur.left > 0) {
      const AttnPiece p = next_piece(a.b, sh, cur);
      auto live_at = [&](int t) {
        const int j = (p.u.t0 + t) * kAttnTK + pl * box_rows;
        return t < p.tb && lane < boxes && j < p.u.hi && j + box_rows > p.u.lo;
      };
      auto page_at = [&](int t) {
        return live_at(t) ? page_of(a.b, p.s, (p.u.t0 + t) * kAttnTK + pl * box_rows) : 0;
      };
      auto copy = [&](int t, int page, bool v) {
        const bool live = live_at(t);
        const uint32_t bytes = box_bytes * __popc(__ballot_sync(0xffffffffu, live));
        if (!wait(emptyb(rg.slot), rg.phase ^ 1u)) return false;
        if (lane == 0) mbar_expect_tx(fullb(rg.slot), bytes);
        __syncwarp();
        if (live)
          tma_load_4d((FP8 ? codes + rg.slot * T::kRawTile : ring + rg.slot * T::kTile) +
                          part * kHalf + pl * box_bytes,
                      v ? &maps.v : &maps.k, fullb(rg.slot), part * 64,
                      ((p.u.t0 + t) * kAttnTK + pl * box_rows) & (ps - 1), p.head, page);
        ++issued;
        rg.next(kN);
        return true;
      };
      int page = page_at(p.ta), next = page_at(p.ta + 1);
      ok = copy(p.ta, page, false);
      for (int t = p.ta; ok && t < p.tb; ++t) {
        const int after = page_at(t + 2);
        if (t + 1 < p.tb) ok = copy(t + 1, next, false);
        if (ok) ok = copy(t, page, true);
        page = next;
        next = after;
      }
    }
    if (*abort_flag && lane == 0)  // let what is in flight land before the CTA can exit
      for (uint32_t j = issued > kN ? issued - kN : 0; j < issued; ++j)
        land(fullb(j % kN), (j / kN) & 1u);
    __syncwarp();
  } else if (FP8 && warp >= kTcCvtWarp) {
    // ------------------------------------------------------------ codes to f16
    const int row0 = threadIdx.x - 32 * kTcCvtWarp;
    Ring rq{0, 0}, rg{0, 0};
    bool ok = true;
    auto convert = [&](const AttnPiece& p, int t, bool v) {
      if (!wait(raw_full(rq.slot), rq.phase) ||
          !wait(empty(rg.slot), rg.phase ^ 1u))
        return false;
      const uint32_t src = codes + rq.slot * T::kRawTile;
#pragma unroll 1
      for (int row = row0; row < kAttnTK; row += 32 * kTcCvtWarps) {
        uint4 w[D / 16];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t off = row * T::kRawPitch + c * 16;
          w[c] = lds128(src + (off ^ ((off >> 3) & T::kRawSwz)));
        }
        const int j = (p.u.t0 + t) * kAttnTK + row;
        if (v && (j < p.u.lo || j >= p.u.hi)) {  // no row attends it: 0, whatever the page holds
#pragma unroll
          for (int c = 0; c < D / 16; ++c) w[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t dst = ring + rg.slot * T::kTile + row * 128u;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t in[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) e4m3x4_f16(in[i], o[2 * i], o[2 * i + 1]);
          const uint32_t at = dst + (c / 4) * kHalf;
          sts128(at + ((((2 * c) & 7) ^ (row & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
          sts128(at + ((((2 * c + 1) & 7) ^ (row & 7)) << 4), make_uint4(o[4], o[5], o[6], o[7]));
        }
      }
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(raw_empty(rq.slot));
        mbar_arrive(full(rg.slot));
      }
      rq.next(T::kRaw);
      rg.next(T::kStages);
      return true;
    };
    while (ok && cur.left > 0) {
      const AttnPiece p = next_piece(a.b, sh, cur);
      ok = convert(p, p.ta, false);
      for (int t = p.ta; ok && t < p.tb; ++t) {
        if (t + 1 < p.tb) ok = convert(p, t + 1, false);
        if (ok) ok = convert(p, t, true);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTcMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool FP8, int D>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t stream) {
  using T = Tc<FP8, D>;
  static int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    const cudaError_t e = cudaFuncSetAttribute(
        attn_tc_kernel<FP8, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)T::kSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  TcMaps maps;
  if (!make_cache_map(&maps.k, a.c.k, a) || !make_cache_map(&maps.v, a.c.v, a))
    return cudaErrorInvalidValue;
  AttnShape sh;
  sh.G = a.hq / a.hkv;
  sh.hkv = a.hkv;
  sh.BR = kTcBR;
  sh.TK = kAttnTK;
  sh.causal = a.causal;
  sh.window = a.window;
  const int ctas = num_sms() < kAttnMaxCtas ? num_sms() : kAttnMaxCtas;
  const cudaError_t e = launch_kernel(attn_tc_kernel<FP8, D>, dim3(ctas), dim3(T::kThreads),
                                      T::kSmem, stream, maps, a, sh);
  if (e != cudaSuccess) return e;
  return launch_attn_join(a, sh, ctas, stream);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t stream) {
  if (a.fp8)
    return a.D == 64 ? launch_typed<true, 64>(a, stream) : launch_typed<true, 128>(a, stream);
  return a.D == 64 ? launch_typed<false, 64>(a, stream) : launch_typed<false, 128>(a, stream);
}

}  // namespace gbmoe
