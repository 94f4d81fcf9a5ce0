// Paged attention of few query rows per kv head (single tokens, short drafts): units of 8 or 16
// rows (token, query head of the group), bound by reading K and V once from HBM.
//
// One persistent CTA per SM takes an equal share of all sequences' key tiles (attn_plan.h). Warp
// 8 streams tiles of 128 keys through a ring of shared-memory stages with TMA, one box per page
// and 128 bytes of the head, 128-byte swizzled; the page ids of a tile are fetched one tile
// ahead. Warps 0..7 own 16 keys of every tile each, with a running maximum, sum and O of their
// own, so that no tile needs a barrier between warps; they are joined through shared memory at
// the end of a piece. Keys and columns lie on the M side of mma.m16n8k16 and the rows on its N
// side, which 8 rows fill:
//   S^T = K Q^T (16 keys x 8 rows, fp32), p = 2^(s - m), O^T += V^T P^T (16 columns x 8 rows).
// Such a product leaves the tensor cores almost idle whatever form it takes, and this one needs
// neither tensor memory nor a trip of P through shared memory (movmatrix turns it). With the
// rows on M instead, half of every product was padding and the e4m3 cache ran at 3.0 TB/s.
// Where a tile is 16 KB (e4m3, or 64 columns) the warps take two at a time: the chain of product,
// maximum, weights, product of one takes longer than HBM takes for the tile.
//
// A unit that the cut between CTAs crosses is joined by the CTA that finishes last (a counter per
// unit, returned to zero), in the pieces' order: the result does not depend on who that is.
//
// bf16 cache: bf16 products, P rounded to bf16. e4m3 cache: codes become f16 (exact) and the
// products run in f16 with Q rounded (saturating) and P rounded to f16; the scales of k and v
// are applied to the scores and to the output. f16 ends at 2^-24 and 2^16, so the maximum that sets
// a row's reference gets a weight of 2^10 and O is rescaled when one would pass 2^14: N keys lose
// at most N 2^-35 of the largest weight. With a largest weight of 1 a tail of 150,000 keys 17.5
// nats below one key was lost where the two met in a warp, 0.4 % of the sum.
#include <cuda_fp16.h>

#include "attn.cuh"

namespace gbmoe {
namespace {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * (kDecWarps + 1);

// NT: rows per unit / 8
template <bool FP8, int D, int NT>
struct Dec {
  static constexpr int kBR = 8 * NT;
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kPitch = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a box row
  static constexpr int kParts = kRowBytes / kPitch;                 // boxes across a row
  static constexpr uint32_t kStage = kAttnTK * kRowBytes;           // one K or V tile
  static constexpr uint32_t kRing = (NT == 1 ? 192 : 160) * 1024;
  static constexpr int kStages = kRing / kStage < 12 ? kRing / kStage : 12;
  static constexpr uint32_t kSwz = kPitch == 128 ? 0x70u : 0x30u;
  static constexpr int kAtOnce = kStages >= 8 ? 2 : 1;              // tiles per softmax step
  // log2 of the weight of the maximum that sets a row's reference, and of the largest
  static constexpr float kLift = FP8 ? 10.f : 0.f, kMost = FP8 ? 14.f : 0.f;
  static constexpr int kJoinPitch = D + (NT == 1 ? 4 : 0);          // floats (4: no conflicts)
  static constexpr uint32_t kJoin = kDecWarps * kBR * kJoinPitch * 4;
  static constexpr uint32_t kTail = NT == 1 ? 1024 : 2048;          // barriers, row sums
  static constexpr size_t kSmem = 1024 + kRing + kJoin + kTail;
  static_assert(kSmem <= 232448, "shared memory per CTA exceeded");
  static_assert((kAttnMaxSeqs + 1) * 4 <= kRing, "the plan lies in the ring");
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
// Four e4m3 bytes as two f16 pairs (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
}
// Transposes an 8x8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t turn(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
// The reference of a row whose maximum is m (log2 units): weights are 2^(s - reference). Scores past
// 2^22 leave the subtraction too few bits to keep weights below 2^16.
__device__ __forceinline__ float lowered(float m, float lift) {
  return lift > 0.f && fabsf(m) < 4194304.f ? m - lift : m;
}
// Spin (bounded) until a copy in flight has landed, so that the CTA does not exit under it.
__device__ __noinline__ void land(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 10000000ull) return;
}

// Pieces of a cut unit whose loads are in flight together: one sequence of 200,000 keys and one kv
// head, cut into 152, takes 34 us with 16 and 38 with 8.
constexpr int kJoinAtOnce = 16;

// A unit that a cut crosses: its rows (row r0 + r of a kv head of a sequence), and the CTAs that
// hold its pieces.
struct CutUnit {
  int q0, head, r0, rows, c0, c1;
};
// What warp 0 lays out for all consumer warps: the next piece (s < 0: none) and the cut units so
// far, the CTA's first if it was begun before it and its last if it is left to the next.
struct DecPlan {
  AttnPiece next;
  int cuts;
  CutUnit cut[2];
};

struct DecMaps {
  CUtensorMap k, v;
};

template <bool FP8, int D, int NT>
__global__ void __launch_bounds__(kDecThreads, 1)
    attn_decode_kernel(const __grid_constant__ DecMaps maps, const __grid_constant__ AttnArgs a,
                       const __grid_constant__ AttnShape sh) {
  using T = Dec<FP8, D, NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw0);
  float* join = reinterpret_cast<float*>(smem + T::kRing);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::kRing + T::kJoin);
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (12 + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 24);
  float2* wml = reinterpret_cast<float2*>(bars + 26);  // [rows][warps]
  int* wsum = reinterpret_cast<int*>(bars + 26 + T::kBR * kDecWarps);  // 32
  DecPlan* plan = reinterpret_cast<DecPlan*>(bars + 42 + T::kBR * kDecWarps);
  static_assert((42 + T::kBR * kDecWarps) * 8 + sizeof(DecPlan) <= T::kTail, "tail");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  AttnSpan span;
  AttnWalk cur;
  const bool quick = quick_plan(a.b, sh);
  if (!quick) {
    // the line of tiles is laid out in the ring before the first copy lands there
    cur = attn_plan(a.b, sh, reinterpret_cast<int*>(smem), wsum, span);
    fence_async_proxy();
  }
  __syncthreads();
  if (quick && (warp == 0 || warp == kDecWarps)) cur = attn_plan_warp(a.b, sh, span);
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
    const AttnScratch sc = attn_scratch(a.scratch, T::kBR);
    const int g = lane >> 2, c = lane & 3;
    uint32_t at = 0;  // ring position of the next tile's K
    auto swz = [](uint32_t off) { return off ^ ((off >> 3) & T::kSwz); };
    auto write_out = [&](int q0, int head, int rr, int d, const float4& v, float M, float L) {
      const int tok = div_group(sh, rr);
      const size_t orow = (size_t)(q0 + tok) * a.hq + head * sh.G + (rr - tok * sh.G);
      const float inv = L == 0.f ? 0.f : a.v_scale / L;  // no key: zeros
      uint2 w;
      w.x = pack_bf16x2(v.x * inv, v.y * inv);
      w.y = pack_bf16x2(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + d) = w;
      if (a.lse && d == 0)
        a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    };
    auto rows_of = [&](const AttnPiece& x) {
      return min(T::kBR, x.q.n * sh.G - x.rb * T::kBR);
    };
    // Warp 0 works the next piece out and fetches its queries into the join area, which is idle
    // while a piece's tiles are worked through: with the ring full of copies in flight a load
    // takes up to 4 us, and a piece that began by loading its queries cost as much.
    constexpr uint32_t kQPitch = 2 * D + 16;
    static_assert(T::kBR * kQPitch <= T::kJoin, "queries");
    int place = 0;  // of the unit's first tile on the line
    auto prepare = [&] {
      AttnPiece next;
      if (!next_piece(a.b, sh, cur, next)) next.s = -1;
      if (next.s >= 0) {
        const uint32_t at = smem_addr(join);
        const int r0 = next.rb * T::kBR;
        for (int i = lane; i < rows_of(next) * (D / 8); i += 32) {
          const int r = i / (D / 8), x = i % (D / 8), tok = div_group(sh, r0 + r);
          cp_async16(at + r * kQPitch + 16 * x,
                     static_cast<const __nv_bfloat16*>(a.q) +
                         (size_t)(next.q.q0 + tok) * a.q_stride +
                         (size_t)(next.head * sh.G + (r0 + r - tok * sh.G)) * D + 8 * x);
        }
      }
      if (lane == 0) plan->next = next;
      place = span.end - cur.left - next.tb;
    };
    // Lane 0 of warp 0 notes the piece p, whose unit's first tile lies at `place`.
    auto note = [&](const AttnPiece& p) {
      if (p.whole()) return;
      CutUnit& x = plan->cut[plan->cuts++];
      x.q0 = p.q.q0;
      x.head = p.head;
      x.r0 = p.rb * T::kBR;
      x.rows = rows_of(p);
      x.c0 = cta_of(span, place);
      x.c1 = cta_of(span, place + p.u.tiles - 1);
    };
    // this lane's query columns of row 8 n + lane / 4, as the B side of the products: two
    // pairs of each 16 columns
    uint32_t qf[NT][D / 16][2];
    bool ok = true;
    // The prepared piece and its queries; p.s < 0 when there is none, ok false after a failure.
    auto take = [&](AttnPiece& p) {
      if (warp == 0) asm volatile("cp.async.wait_all;" ::: "memory");
      if (consumers_sync(!ok)) ok = false;
      if (!ok) return;
      p = plan->next;
      if (p.s < 0) return;
      const int rows = rows_of(p);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(join) + (8 * n + g) * kQPitch;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t lo = 0u, hi = 0u;
          if (8 * n + g < rows && FP8) {
            // e4m3 fragments hold columns 4c .. 4c + 3 of each 16: Q's follow that order
            const uint2 w = *reinterpret_cast<const uint2*>(src + 32 * k + 8 * c);
            const float2 x = unpack_bf16x2(w.x), y = unpack_bf16x2(w.y);
            auto cut = [](float v) { return v > 65504.f ? 65504.f : (v < -65504.f ? -65504.f : v); };
            lo = pack_f16x2(cut(x.x), cut(x.y));
            hi = pack_f16x2(cut(y.x), cut(y.y));
          } else if (8 * n + g < rows) {
            lo = *reinterpret_cast<const uint32_t*>(src + 32 * k + 4 * c);
            hi = *reinterpret_cast<const uint32_t*>(src + 32 * k + 16 + 4 * c);
          }
          qf[n][k][0] = lo;
          qf[n][k][1] = hi;
        }
      }
    };
    AttnPiece p;
    if (threadIdx.x == 0) plan->cuts = 0;
    if (warp == 0) prepare();
    take(p);
    consumers_sync(false);  // the queries are read
    while (ok && p.s >= 0) {
      if (warp == 0) {
        if (lane == 0) note(p);
        prepare();
      }
      const int rows = rows_of(p);
      // the keys of this lane's rows 8 n + 2 c + e; those that every row attends need no mask
      KeyRange kr[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * c + e;
          kr[n][e] = key_range(p.q, div_group(sh, p.rb * T::kBR + r), sh.causal, sh.window);
          if (r >= rows) kr[n][e].hi = kr[n][e].lo = 0;
        }
      const KeyRange k0 = key_range(p.q, p.u.i0, sh.causal, sh.window);
      const KeyRange k1 = key_range(p.q, p.u.i1, sh.causal, sh.window);
      float o[NT][D / 16][4];  // (column 16 i + g, row 2 c), (.., row 2 c + 1), (column + 8, ..)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
      float m[NT][2], l[NT][2];  // m: the reference of the weights, log2 units
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
      }

      for (int t = p.ta; ok && t < p.tb; t += T::kAtOnce) {
        const int count = min(T::kAtOnce, p.tb - t);
        // tile t + u: K in ring position at + 2 u, V in the next; this warp's keys from j0 + 128 u
        const int j0 = (p.u.t0 + t) * kAttnTK + warp * 16;
        auto some = [&](int u) {
          return u < count && j0 + kAttnTK * u < p.u.hi && j0 + kAttnTK * u + 16 > p.u.lo;
        };
        auto slot = [&](uint32_t pos) { return pos % T::kStages; };
        auto filled = [&](uint32_t pos) {
          return wait_fast(full(slot(pos)), pos / T::kStages & 1u, abort_flag, status);
        };
        auto release = [&](uint32_t pos) {
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(slot(pos)));
        };
        // S^T: (key g, row 2 c), (key g, row 2 c + 1), (key g + 8, ..)
        float s[T::kAtOnce][NT][4];
#pragma unroll
        for (int u = 0; u < T::kAtOnce; ++u) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[u][n][j] = 0.f;
          if (u < count && !filled(at + 2 * u)) {
            ok = false;
            break;
          }
        }
        if (!ok) break;
        // the tiles' products in turn: each is a chain of sums. A tile that has none of this
        // warp's keys is worked through as well, whatever its stage holds: its scores drop out
        const uint32_t row = warp * 16 + (lane & 15);
#pragma unroll
        for (int k = 0; k < D / (FP8 ? 32 : 16); ++k)
#pragma unroll
          for (int u = 0; u < T::kAtOnce; ++u) {
            const uint32_t st = base + slot(at + 2 * u) * T::kStage;
            uint32_t w[4];
            if (FP8) {
              // keys 0-7 and 8-15 x 32 columns, 16 bytes per row of an 8x8 matrix
              uint32_t f[2][4];
              ldsm4(st + swz(row * T::kPitch + k * 32 + (lane >> 4) * 16), w);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                e4m3x4_f16(w[2 * h], f[h][0], f[h][2]);
                e4m3x4_f16(w[2 * h + 1], f[h][1], f[h][3]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma16816<true>(s[u][n], f[h], qf[n][2 * k + h][0], qf[n][2 * k + h][1]);
              }
            } else {
              const uint32_t col = (k % 4) * 32 + (lane >> 4) * 16;
              ldsm4(st + (k / 4) * (kAttnTK * 128) + swz(row * 128 + col), w);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816<false>(s[u][n], w, qf[n][k][0], qf[n][k][1]);
            }
          }
#pragma unroll
        for (int u = 0; u < T::kAtOnce; ++u)
          if (u < count) release(at + 2 * u);
        // scores in log2 units; keys that a row does not attend drop out
        float mn[NT][2];
        bool grows = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float most[2] = {m[n][0] + T::kMost, m[n][1] + T::kMost};
          mn[n][0] = most[0];
          mn[n][1] = most[1];
#pragma unroll
          for (int u = 0; u < T::kAtOnce; ++u) {
            const int ju = j0 + kAttnTK * u;
            const bool mask =
                u >= count || ju < max(k0.lo, k1.lo) || ju + 16 > min(k0.hi, k1.hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v = s[u][n][e] * a.scale_log2;
              if (mask) {
                const int j = ju + g + 8 * (e >> 1);
                if (u >= count || j < kr[n][e & 1].lo || j >= kr[n][e & 1].hi) v = -INFINITY;
              }
              s[u][n][e] = v;
              mn[n][e & 1] = fmaxf(mn[n][e & 1], v);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
              mn[n][e] = fmaxf(mn[n][e], __shfl_xor_sync(0xffffffffu, mn[n][e], x));
            grows |= mn[n][e] > most[e];
          }
        }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (FP8)
                mn[n][e] = mn[n][e] > m[n][e] + T::kMost ? lowered(mn[n][e], T::kLift) : m[n][e];
              const float f = mn[n][e] > m[n][e] ? ex2(m[n][e] - mn[n][e]) : 1.f;
              m[n][e] = mn[n][e];
              l[n][e] *= f;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[n][i][e] *= f;
                o[n][i][2 + e] *= f;
              }
            }
        }
        uint32_t pf[T::kAtOnce][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
          const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
          for (int u = 0; u < T::kAtOnce; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = ex2(s[u][n][2 * h] - m0), y = ex2(s[u][n][2 * h + 1] - m1);
              l[n][0] += x;
              l[n][1] += y;
              pf[u][n][h] = turn(pack16<FP8>(x, y));
            }
        }
#pragma unroll
        for (int u = 0; u < T::kAtOnce; ++u) {
          if (u >= count) continue;
          const uint32_t pos = at + 2 * u + 1;
          if (!filled(pos)) {
            ok = false;
            break;
          }
          if (some(u)) {
            const uint32_t st = base + slot(pos) * T::kStage;
            const int ju = j0 + kAttnTK * u;
            if (ju < p.u.lo || ju + 16 > p.u.hi) {
              // v of positions that no row attends: 0, whatever the page holds (0 * NaN = NaN)
              for (int i = lane; i < 16 * (T::kRowBytes / 16); i += 32) {
                const int r = i / (T::kRowBytes / 16), x = i % (T::kRowBytes / 16);
                if (ju + r < p.u.lo || ju + r >= p.u.hi)
                  sts128(st + (x * 16 / T::kPitch) * (kAttnTK * T::kPitch) +
                             (warp * 16 + r) * T::kPitch + x * 16 % T::kPitch,
                         make_uint4(0u, 0u, 0u, 0u));
              }
              __syncwarp();
              fence_async_proxy();  // before the stage's next copy
            }
            if (FP8) {
              // transposed 8x8 matrices of byte pairs: columns 2 g and 2 g + 1 of two keys a word
              const uint32_t row = warp * 16 + (lane & 15);
#pragma unroll
              for (int k = 0; k < D / 32; ++k) {
                uint32_t w[4], f[4];
                ldsm4t(st + swz(row * T::kPitch + k * 32 + (lane >> 4) * 16), w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  e4m3x4_f16(__byte_perm(w[2 * h], 0u, 0x3120), f[0], f[1]);
                  e4m3x4_f16(__byte_perm(w[2 * h + 1], 0u, 0x3120), f[2], f[3]);
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    mma16816<true>(o[n][2 * k + h], f, pf[u][n][0], pf[u][n][1]);
                }
              }
            } else {
              // matrices: keys 0-7 x columns 0-7, keys 0-7 x 8-15, keys 8-15 x 0-7, x 8-15
              const uint32_t row = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                uint32_t w[4];
                const uint32_t col = (k % 4) * 32 + ((lane >> 3) & 1) * 16;
                ldsm4t(st + (k / 4) * (kAttnTK * 128) + swz(row * 128 + col), w);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma16816<false>(o[n][k], w, pf[u][n][0], pf[u][n][1]);
              }
            }
          }
          release(pos);
        }
        at += 2 * count;
      }

      // ---------------------------------------------------------- the piece's result
      AttnPiece next;
      take(next);
      if (!ok) break;
      consumers_sync(false);  // the queries are read
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
          const int r = 8 * n + 2 * c + e;
          if (g == 0) wml[r * kDecWarps + warp] = make_float2(m[n][e], l[n][e]);
          if (r < rows) {
            float* dst = join + (warp * T::kBR + r) * T::kJoinPitch;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              if (FP8) {  // columns 2 g and 2 g + 1 of the 16
                *reinterpret_cast<float2*>(dst + 16 * i + 2 * g) =
                    make_float2(o[n][i][e], o[n][i][2 + e]);
              } else {
                dst[16 * i + g] = o[n][i][e];
                dst[16 * i + 8 + g] = o[n][i][2 + e];
              }
            }
          }
        }
      consumers_sync(false);
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
          const float4 x = *reinterpret_cast<const float4*>(join + (w * T::kBR + r) * T::kJoinPitch + d);
          L = fmaf(f, ml[w].y, L);
          v.x = fmaf(f, x.x, v.x);
          v.y = fmaf(f, x.y, v.y);
          v.z = fmaf(f, x.z, v.z);
          v.w = fmaf(f, x.w, v.w);
        }
        if (p.whole()) {
          write_out(p.q.q0, p.head, p.rb * T::kBR + r, d, v, M, L);
        } else {
          const size_t row = (size_t)slot_out * T::kBR + r;
          *reinterpret_cast<float4*>(sc.o + row * D + d) = v;
          if (d == 0) sc.ml[row] = make_float2(M, L);
        }
      }
      p = next;
      consumers_sync(false);  // the join area is free again
    }
    // Cut units are joined by the CTA that finishes last: both are counted here, so that a piece
    // that ends in the middle of the CTA's range waits for no fence and no atomic.
    const int cuts = ok ? plan->cuts : 0;
    if (cuts) {
      if ((int)threadIdx.x < cuts) {  // all warps' stores lie behind a barrier
        const CutUnit x = plan->cut[threadIdx.x];
        __threadfence();
        const bool last = atomicAdd(a.counters + x.c0, 1) == x.c1 - x.c0;
        if (last) atomicExch(a.counters + x.c0, 0);
        __threadfence();
        wsum[threadIdx.x] = last;
      }
      consumers_sync(false);
      for (int k = 0; k < cuts; ++k) {
        if (!wsum[k]) continue;
        const CutUnit x = plan->cut[k];
        for (int i = threadIdx.x; i < x.rows * (D / 4); i += 32 * kDecWarps) {
          const int r = i / (D / 4), d = i % (D / 4) * 4;
          float M = -INFINITY, L = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c = x.c0; c <= x.c1; c += kJoinAtOnce) {
            float2 ml[kJoinAtOnce];
            float4 y[kJoinAtOnce];
#pragma unroll
            for (int j = 0; j < kJoinAtOnce; ++j) {
              const int cj = min(c + j, x.c1);
              const size_t row = (size_t)(cj == x.c0 ? 2 * cj + 1 : 2 * cj) * T::kBR + r;
              ml[j] = __ldcg(sc.ml + row);
              y[j] = __ldcg(reinterpret_cast<const float4*>(sc.o + row * D + d));
            }
            float mx = M;
#pragma unroll
            for (int j = 0; j < kJoinAtOnce; ++j) {
              if (c + j > x.c1) ml[j] = make_float2(-INFINITY, 0.f);
              mx = fmaxf(mx, ml[j].x);
            }
            const float ms = mx == -INFINITY ? 0.f : mx;
            const float f0 = ex2(M - ms);
            M = mx;
            L *= f0;
            v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
#pragma unroll
            for (int j = 0; j < kJoinAtOnce; ++j) {
              const float f = ex2(ml[j].x - ms);
              L = fmaf(f, ml[j].y, L);
              v.x = fmaf(f, y[j].x, v.x);
              v.y = fmaf(f, y[j].y, v.y);
              v.z = fmaf(f, y[j].z, v.z);
              v.w = fmaf(f, y[j].w, v.w);
            }
          }
          write_out(x.q0, x.head, x.r0 + r, d, v, M, L);
        }
      }
    }
  }
  __syncthreads();
}

template <bool FP8, int D, int NT>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t stream) {
  using T = Dec<FP8, D, NT>;
  static int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    const cudaError_t e = cudaFuncSetAttribute(
        attn_decode_kernel<FP8, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)T::kSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  DecMaps maps;
  if (!make_cache_map(&maps.k, a.c.k, a) || !make_cache_map(&maps.v, a.c.v, a))
    return cudaErrorInvalidValue;
  const int ctas = num_sms() < kAttnMaxCtas ? num_sms() : kAttnMaxCtas;
  const bool few = (long long)a.b.S * a.hkv < ctas;
  constexpr int kShift = NT == 1 ? 3 : 4;
  const AttnShape sh = attn_shape(a, kShift, unit_cost(kShift, D, FP8, few));
  static_assert(T::kBR == 1 << kShift, "rows per unit");
  static_assert(AttnShape::half == 1 && AttnShape::full == 1,
                "a cut unit's CTAs are counted as neighbours");
  return launch_kernel(attn_decode_kernel<FP8, D, NT>, dim3(ctas), dim3(kDecThreads), T::kSmem,
                       stream, maps, a, sh);
}
template <int NT>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream) {
  if (a.fp8)
    return a.D == 64 ? launch_typed<true, 64, NT>(a, stream) : launch_typed<true, 128, NT>(a, stream);
  return a.D == 64 ? launch_typed<false, 64, NT>(a, stream) : launch_typed<false, 128, NT>(a, stream);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs& a, bool eight, cudaStream_t stream) {
  return eight ? launch_rows<1>(a, stream) : launch_rows<2>(a, stream);
}

}  // namespace gbmoe
