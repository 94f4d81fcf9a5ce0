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
// m is the maximum of the row's first keys and is kept until a tile's maximum lies far above it
// (kSlack: weights of 2^60 in bf16 and fp32 lose nothing against weights of 1): only then is O
// rescaled in tensor memory, and no tile waits for its own maximum. f16 weights (e4m3 cache) end at
// 2^-24 and 2^16, so the maximum that sets the reference gets 2^7 (kLift), and N keys lose at most
// N 2^-32 of the largest weight. 8191 tokens: 364 us with 2^0 and 2^7, 369 with 2^8, 394 with 2^9,
// which leaves less room before O is rescaled. P is handed over in two steps
// of 64 keys, so that the second product begins while the second half is still being weighed.
//
//   warps 0-3, 4-7   softmax of half 0 / 1; they also bring the unit's Q into shared memory (the
//                    next piece's while the last product runs) and write the piece's result
//   warp 8           MMA issue (one elected thread)
//   warp 9           the schedule, as a ring of piece descriptors ahead of the other roles, and
//                    the tile copies: TMA, one box per page and 128 bytes of the head; page ids
//                    a tile ahead, the next piece's Q into L2
//   warp 11          bf16 cache in pages below 64 rows: V's copies (a tile in pages of 16 rows
//                    takes 16 boxes, which one warp issues one after the other)
//   warp 10          bf16 cache: zeroes what a V tile holds outside the unit's keys
//   warps 10, 11     e4m3 cache: codes to f16 (exact) into the operand tiles
//
// Tensor memory: S/P of half h at columns 128 h, O of half h at 256 + 128 h; heads of 64: S at
// 128 h, P at 256 + 64 h, O at 384 + 64 h. Operand order in
// the ring: K0, V0, K1, V1, ...; the scores of the next tile are issued ahead of a tile's second
// product. bf16 cache: bf16 products; e4m3: f16 products with Q rounded to f16 (saturating).
//
// Bound by the tensor cores: a tile of both halves is 2048 cycles of products (heads of 128), and
// a long prompt's steady step takes 2550 to 2700; the products alone, without a softmax, 2360.
// 8191 causal tokens of 32 + 8 heads: 347 us, 1585 TFLOP/s (0.83 of the measured bf16 rate).
// 64 + 8 heads of 64: 552 us, bound by the softmax, whose work does not halve with the products
// (626 with P over the scores, as for 128). e4m3 (32 + 8 heads of 128): 364 us, bound by the two
// warps that turn codes to f16.
// Beginning a piece costs about 2 us (drain of the last O, first scores), which packed prompts
// feel: 5955 tokens of 5 sequences 85 us, 896 TFLOP/s. Two issuing threads, one per half, took
// 459 us for the long prompt: the halves' products then alternate on the tensor core and none
// finishes early.
#include <cuda_fp16.h>

#include "attn.cuh"

namespace gbmoe {
namespace {

constexpr int kTcBR = 256;
constexpr int kTcMmaWarp = 8, kTcCopyWarp = 9, kTcCvtWarp = 10, kTcCopyWarpV = 11;
constexpr int kTcCvtWarps = 2;
constexpr int kTcSplitShift = 6;  // pages below 1 << 6 rows: K's and V's copies by a warp each

template <bool FP8, int D>
struct Tc {
  static constexpr int kThreads = 32 * 12;                  // three warps a scheduler
  static constexpr uint32_t kTile = kAttnTK * D * 2;        // one operand tile (16 bit)
  static constexpr uint32_t kRawTile = kAttnTK * D;         // one tile of codes
  static constexpr int kRaw = FP8 ? 3 : 0;                  // code stages
  static constexpr int kStages = FP8 ? 3 : 4;               // operand stages
  // Tensor memory columns of a half: its scores, weights and output. With 64 columns of output the
  // weights have a place of their own and the next tile's scores need not wait for their product.
  static constexpr bool kApart = D == 64;
  static __host__ __device__ constexpr uint32_t s_col(int g) { return 128u * g; }
  static __host__ __device__ constexpr uint32_t p_col(int g) { return kApart ? 256u + 64u * g : 128u * g; }
  static __host__ __device__ constexpr uint32_t o_col(int g) {
    return kApart ? 384u + 64u * g : 256u + 128u * g;
  }
  static constexpr int kOutCols = 32;                       // columns staged at a time
  static constexpr uint32_t kOut = 2 * 128 * kOutCols * 2;  // staging of the output rows
  static constexpr uint32_t kQ = 2 * kTile;
  // log2 of the weight that the maximum gets when it sets the reference, and of the largest weight
  // before O is rescaled: bf16 has fp32's range, f16 ends at 2^16
  static constexpr float kLift = FP8 ? 7.f : 0.f;
  static constexpr float kSlack = FP8 ? 14.f : 60.f;
  static constexpr uint32_t kRawPitch = D < 128 ? D : 128;  // bytes of a code row
  static constexpr uint32_t kRawSwz = kRawPitch == 128 ? 0x70u : 0x30u;
  using Shape = AttnTcShape<D>;
  static_assert(Shape::full == tile_cost(8, D), "one cost");
  static constexpr int kReaders = 8 + 1 + 2;  // warps that read a piece: softmax, MMA, 10 and 11
  static constexpr size_t kSmem = 1024 + kQ + kStages * kTile + kRaw * kRawTile + kOut + 1024;
  static_assert(kSmem <= 232448, "shared memory per CTA exceeded");
  static_assert((kAttnMaxSeqs + 1) * 4 <= kQ + kStages * kTile, "the plan lies in Q and the ring");
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
__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// Two fp32 values in one 64-bit register, and the packed operations on them.
__device__ __forceinline__ uint64_t pair_bits(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint64_t pair(float x, float y) {
  return pair_bits(__float_as_uint(x), __float_as_uint(y));
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Spin (bounded) until a copy in flight has landed, so that the CTA does not exit under it.
__device__ __noinline__ void land(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 10000000ull) return;
}

// One thread of the converged warp; the compiler knows that there is one, so that operands of
// the instructions it issues stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(p));
  return p != 0;
}

struct TcMaps {
  CUtensorMap k, v;
};

// A piece as the schedule publishes it.
struct alignas(16) TcPiece {
  int nt;              // tiles; 0: no piece is left
  int j0;              // first key of the first tile
  int lo, hi;          // keys that any row of the unit attends
  int in_lo, in_hi;    // keys that every row attends
  int rows, r0;        // rows of the unit, its first row in the sequence
  int q0, n, L, head;  // the sequence, the kv head
  int slot;            // piece slot in the workspace, -1: the whole unit
  int seq;             // index of the sequence
  int pad[2];
};
static_assert(sizeof(TcPiece) == 64, "read as four 16-byte words");
constexpr int kTcPieces = 4;

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
                   const __grid_constant__ typename Tc<FP8, D>::Shape sh) {
  using T = Tc<FP8, D>;
  constexpr uint32_t kHalf = kAttnTK * 128;  // a 64-column half of an operand tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw0);
  const uint32_t q_base = base, ring = base + T::kQ, codes = ring + T::kStages * T::kTile;
  const uint32_t outs = codes + T::kRaw * T::kRawTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (outs - base) + T::kOut);
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };           // operand stage filled
  auto empty = [&](int s) { return bar0 + 8u * (5 + s); };    // ... and read by its MMAs
  auto q_full = [&](int g) { return bar0 + 8u * (10 + g); };
  auto s_full = [&](int g) { return bar0 + 8u * (12 + g); };
  auto p_full = [&](int g, int h) { return bar0 + 8u * (h ? 32 + g : 14 + g); };  // 64 keys each
  auto pv_done = [&](int g) { return bar0 + 8u * (16 + g); };
  auto raw_full = [&](int s) { return bar0 + 8u * (18 + s); };
  auto raw_empty = [&](int s) { return bar0 + 8u * (22 + s); };
  auto pa_done = [&](int g) { return bar0 + 8u * (42 + g); };  // first 64 keys' product
  auto s_read = [&](int g) { return bar0 + 8u * (44 + g); };   // kApart: scores in registers
  auto v_raw = [&](int s) { return bar0 + 8u * (26 + s); };   // stage s: an edge V tile landed
  auto d_full = [&](int i) { return bar0 + 8u * (34 + i); };  // piece descriptors
  auto d_empty = [&](int i) { return bar0 + 8u * (38 + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 31);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  TcPiece* pieces = reinterpret_cast<TcPiece*>(bars + 46);
  int* wsum = reinterpret_cast<int*>(bars + 46 + kTcPieces * 8);  // 32
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = a.b.status;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(full(s), FP8 ? kTcCvtWarps : 1);
      mbar_init(empty(s), 1);
      mbar_init(v_raw(s), 1);
    }
    for (int s = 0; s < T::kRaw; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), kTcCvtWarps);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(q_full(g), 4);
      mbar_init(s_full(g), 1);
      mbar_init(p_full(g, 0), 4);
      mbar_init(p_full(g, 1), 4);
      mbar_init(pv_done(g), 1);
      mbar_init(pa_done(g), 1);
      mbar_init(s_read(g), 4);
    }
    for (int i = 0; i < kTcPieces; ++i) {
      mbar_init(d_full(i), 1);
      mbar_init(d_empty(i), T::kReaders);
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
  AttnSpan span;
  AttnWalk cur;
  const bool quick = quick_plan(a.b, sh);
  if (!quick) {
    cur = attn_plan(a.b, sh, reinterpret_cast<int*>(smem), wsum, span);
    fence_async_proxy();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (quick && warp == kTcCopyWarp) cur = attn_plan_warp(a.b, sh, span);
  const uint32_t tmem = *tmem_slot;
  // a wait whose answer is the whole warp's (tcgen05 and warp barriers follow it)
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_fast(bar, parity, abort_flag, status)) != 0;
  };
  // the next piece, read by a whole warp (or by one thread for its warp)
  Ring dq{0, 0};
  auto read_piece = [&](TcPiece& p) {
    const int4* src = reinterpret_cast<const int4*>(pieces + dq.slot);
    const int4 w0 = src[0], w1 = src[1], w2 = src[2], w3 = src[3];
    p.nt = w0.x; p.j0 = w0.y; p.lo = w0.z; p.hi = w0.w;
    p.in_lo = w1.x; p.in_hi = w1.y; p.rows = w1.z; p.r0 = w1.w;
    p.q0 = w2.x; p.n = w2.y; p.L = w2.z; p.head = w2.w;
    p.slot = w3.x; p.seq = w3.y;
  };
  auto release_piece = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(d_empty(dq.slot));
    dq.next(kTcPieces);
  };
  auto get_piece = [&](TcPiece& p) {
    if (!wait(d_full(dq.slot), dq.phase)) return false;
    read_piece(p);
    release_piece();
    return p.nt > 0;
  };
  // whether the tile at key j holds positions outside the unit's keys
  auto edge = [](const TcPiece& p, int j) { return j < p.lo || j + kAttnTK > p.hi; };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const AttnScratch sc = attn_scratch(a.scratch, kTcBR);
    const int g = warp >> 2;
    const int row = threadIdx.x & 127;                       // of this half
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + T::s_col(g), tp = tmem + lanes + T::p_col(g),
                   to = tmem + lanes + T::o_col(g);
    const uint32_t q_half = q_base + g * T::kTile;
    constexpr int kLanes = D / 8;  // lanes that a query row takes, 16 bytes each
    // A piece as this thread's row needs it.
    struct Job {
      int nt, j0;          // tiles, first key of the first
      int lo, hi;          // the row's keys
      int in_lo, in_hi;    // keys that every row of the unit attends
      int row;             // output row (token * heads + head), or the slot's; -1: no such row
      bool whole;
    } job;
    // Moves to the next piece that has rows in this half: 1, 0 when none is left, or, unless
    // `block`, 2 when the schedule has not got there (it may be waiting for this very tile's
    // weights).
    auto seek = [&](bool block) {
      for (;;) {
        if (!block && !__all_sync(0xffffffffu, mbar_test_wait(d_full(dq.slot), dq.phase)))
          return 2;
        if (!wait(d_full(dq.slot), dq.phase)) return 0;
        const TcPiece& p = pieces[dq.slot];
        if (p.nt == 0) return 0;
        if (p.rows > 128 * g) return 1;
        release_piece();
      }
    };
    // Sends the warp's query rows of that piece to shared memory (Q's place must be free), D / 8
    // lanes a row so that a copy covers whole rows.
    auto send_q = [&]() {
      const TcPiece& p = pieces[dq.slot];
      const int r = 128 * g + row, rr = p.r0 + r;
      const int tok = div_group(sh, rr), head = p.head * sh.G + (rr - tok * sh.G);
      const unsigned long long src =
          reinterpret_cast<unsigned long long>(a.q) +
          (r < p.rows ? 2ull * ((size_t)(p.q0 + tok) * a.q_stride + (size_t)head * D) : 0ull);
      const uint32_t some = __ballot_sync(0xffffffffu, r < p.rows);
      const int c = lane % kLanes;
      const uint32_t dst = q_half + (c / 8) * kHalf;
#pragma unroll 2
      for (int i = 0; i < kLanes; ++i) {
        const int l = i * (32 / kLanes) + lane / kLanes, r2 = (warp & 3) * 32 + l;
        const unsigned long long at = __shfl_sync(0xffffffffu, src, l) + c * 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         dst + r2 * 128u + (((c & 7) ^ (r2 & 7)) << 4)),
                     "l"(at), "r"((some >> l) & 1u ? 16u : 0u)
                     : "memory");
      }
    };
    // This thread's job in that piece, which is given back to the schedule.
    auto take_job = [&]() {
      const TcPiece& p = pieces[dq.slot];
      const int r = 128 * g + row, rr = p.r0 + r;
      const bool valid = r < p.rows;
      const int tok = div_group(sh, rr), head = p.head * sh.G + (rr - tok * sh.G);
      const KeyRange kr = key_range(SeqInfo{p.q0, p.n, p.L}, tok, sh.causal, sh.window);
      job.nt = p.nt;
      job.j0 = p.j0;
      job.lo = kr.lo;
      job.hi = valid ? kr.hi : 0;
      job.in_lo = p.in_lo;
      job.in_hi = p.in_hi;
      job.whole = p.slot < 0;
      job.row = !valid ? -1 : job.whole ? (p.q0 + tok) * a.hq + head : p.slot * kTcBR + r;
      release_piece();
    };
    // The query rows have arrived: hand Q to the tensor core.
    auto finish_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (FP8) {  // bf16 to f16 in place, by the thread that copied it
        const int c = lane % kLanes;
#pragma unroll 2
        for (int i = 0; i < kLanes; ++i) {
          const int r2 = (warp & 3) * 32 + i * (32 / kLanes) + lane / kLanes;
          const uint32_t at = q_half + (c / 8) * kHalf + r2 * 128u + (((c & 7) ^ (r2 & 7)) << 4);
          uint4 v = lds128(at);
          v.x = bf16x2_f16(v.x);
          v.y = bf16x2_f16(v.y);
          v.z = bf16x2_f16(v.z);
          v.w = bf16x2_f16(v.w);
          sts128(at, v);
        }
      }
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(g));
    };
    int have = seek(true);
    if (have) {
      send_q();
      finish_q();
    }
    uint32_t tc = 0;  // tiles of this half so far
    const uint64_t sc2 = pair(a.scale_log2, a.scale_log2);
    const float lift = T::kLift / a.scale_log2;  // in units of the raw scores
    while (have) {
      take_job();
      float m = -INFINITY, l = 0.f;   // m: the reference of the weights, raw score units
      bool ok = true;
      have = 2;
      for (int t = 0; t < job.nt; ++t, ++tc) {
        if (!wait(s_full(g), tc & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the last scores are out, so Q's place is free: the next piece's is on its way while
        // this tile is weighed
        if (t + 1 == job.nt && (have = seek(false)) == 1) send_q();
        const int j0 = job.j0 + t * kAttnTK;
        const bool masked = j0 < job.in_lo || j0 + kAttnTK > job.in_hi;
        uint64_t sum[2] = {0ull, 0ull};
        // The tile in two steps of 64 keys; the product over a step's keys may begin before the
        // next step's weights are there.
        uint32_t s[2][32];
#pragma unroll
        for (int i = 0; i < 2; ++i) tmem_ld32(ts + 32 * i, s[i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_wait_ld(s[i]);
          if (T::kApart && h == 1) {  // the next tile's scores may overwrite these
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_read(g));
          }
          auto drop = [&]() {  // keys that this row does not attend
            const int lo = job.lo - j0 - 64 * h, hi = job.hi - j0 - 64 * h;
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              uint32_t& x = s[c / 32][c % 32];
              x = c >= hi ? 0xff800000u : x;  // -inf
            }
            if (j0 < job.in_lo)
#pragma unroll
              for (int c = 0; c < 64; ++c) {
                uint32_t& x = s[c / 32][c % 32];
                x = c < lo ? 0xff800000u : x;
              }
          };
          if (masked) drop();
          // The weights go by the reference so far; the keys' own maximum, off that path, only
          // tells whether they grow too large. A piece's first keys set the reference.
          if (t == 0 && h == 0) {
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 64; c += 2)
              mx[c / 2 & 3] = fmaxf(fmaxf(mx[c / 2 & 3], __uint_as_float(s[c / 32][c % 32])),
                                    __uint_as_float(s[c / 32][c % 32 + 1]));
            m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (FP8) m -= lift;
          }
          uint32_t w[32];
          for (;;) {
            const float off = m == -INFINITY ? 0.f : -m * a.scale_log2;
            const uint64_t off2 = pair(off, off);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            uint64_t part[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const uint32_t u = s[c / 16][2 * c % 32], v = s[c / 16][2 * c % 32 + 1];
              mx[c & 3] = fmaxf(fmaxf(mx[c & 3], __uint_as_float(u)), __uint_as_float(v));
              float e0, e1;
              unpair(fma2(pair_bits(u, v), sc2, off2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              part[c & 1] = add2(part[c & 1], pair(e0, e1));
              w[c] = FP8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
            }
            const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (!__any_sync(0xffffffffu, mn > m && (mn - m) * a.scale_log2 > T::kSlack)) {
              sum[0] = add2(sum[0], part[0]);
              sum[1] = add2(sum[1], part[1]);
              break;
            }
            // O catches up with the new maxima once the product before these keys' is done (a
            // piece's first keys have none, but their reference is their maximum)
            if (!(h ? wait(pa_done(g), tc & 1u) : wait(pv_done(g), (tc - 1) & 1u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float to_m = FP8 ? mn - lift : mn;
            const float f = to_m > m ? ex2((m - to_m) * a.scale_log2) : 1.f;
            m = fmaxf(m, to_m);
            {
              float x, y, u, v;
              unpair(sum[0], x, y);
              unpair(sum[1], u, v);
              l = (l + ((x + y) + (u + v))) * f;
              sum[0] = sum[1] = 0ull;
            }
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              tmem_ld32(to + 32 * i, w);
              tmem_wait_ld(w);
#pragma unroll
              for (int c = 0; c < 32; ++c) w[c] = __float_as_uint(__uint_as_float(w[c]) * f);
              tmem_st32(to + 32 * i, w);
            }
            tmem_wait_st();
          }
          if (!ok) break;
          if (h == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i) tmem_ld32(ts + 64 + 32 * i, s[i]);
          if (T::kApart && h == 0) {  // P's place is free when the last tile's product is done
            if (!wait(pv_done(g), (tc - 1) & 1u)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          tmem_st32(tp + 32 * h, w);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(g, h));
        }
        if (!ok) break;
        float x, y, u, v;
        unpair(sum[0], x, y);
        unpair(sum[1], u, v);
        l += (x + y) + (u + v);
      }
      if (!ok) break;
      if (have == 2 && (have = seek(true)) == 1) send_q();
      if (have) finish_q();
      if (!wait(pv_done(g), (tc - 1) & 1u)) break;
      tc_fence_after();
      const float ml = m == -INFINITY ? -INFINITY : m * a.scale_log2;
      if (job.whole) {
        // through shared memory, kOutCols columns at a time, so that a store covers whole
        // stretches of a row. Rolled: code of a piece's end that is not in the instruction cache
        // costs more than its execution.
        constexpr int kPer = T::kOutCols / 8;  // lanes (16 bytes each) a row
        constexpr uint32_t kPitch = T::kOutCols * 2;
        static_assert(T::kOutCols == 32, "one tensor memory load a pass");
        const uint32_t st = outs + warp * (32 * kPitch);
        const float inv = l == 0.f ? 0.f : a.v_scale / l;
        const int c = lane % kPer;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += T::kOutCols) {
          uint32_t o[32];
          tmem_ld32(to + c0, o);
          tmem_wait_ld(o);
          __syncwarp();  // the columns before have been read
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(o[8 * k + 2 * i]) * inv,
                                 __uint_as_float(o[8 * k + 2 * i + 1]) * inv);
            sts128(st + lane * kPitch + ((k ^ ((lane >> 1) & (kPer - 1))) << 4),
                   make_uint4(w[0], w[1], w[2], w[3]));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int r = i * (32 / kPer) + lane / kPer;
            const int orow = __shfl_sync(0xffffffffu, job.row, r);
            const uint4 v = lds128(st + r * kPitch + ((c ^ ((r >> 1) & (kPer - 1))) << 4));
            if (orow >= 0)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (size_t)orow * D +
                                        c0 + c * 8) = v;
          }
        }
        if (a.lse && job.row >= 0)
          a.lse[job.row] = l == 0.f ? -INFINITY : (ml + log2f(l)) * 0.6931471805599453f;
      } else {
        uint4* dst = reinterpret_cast<uint4*>(sc.o + (size_t)job.row * D);
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(to + 32 * i, o);
          tmem_wait_ld(o);
          if (job.row >= 0)
#pragma unroll
            for (int c = 0; c < 4; ++c) stg256(dst + 8 * i + 2 * c, &o[8 * c]);
        }
        if (job.row >= 0) sc.ml[job.row] = make_float2(ml, l);
      }
      tc_fence_before();
    }
  } else if (warp == kTcMmaWarp) {
    // ------------------------------------------------------------ products (one thread)
    if (elect_one()) {
      constexpr uint32_t kIdS = idesc_attn(FP8, kAttnTK, false), kIdO = idesc_attn(FP8, D, true);
      constexpr uint32_t kStep = T::kTile >> 4;  // descriptor units per stage
      const uint64_t q_half = sdesc_sw128(q_base), k_ring = sdesc_sw128(ring),
                     v_ring = sdesc_v(ring);
      Ring rg{0, 0};
      uint32_t pieces_of = 0;  // bit g: parity of half g's pieces so far
      uint32_t tiles_of = 0;   // ... of its tiles
      auto wait1 = [&](uint32_t bar, uint32_t parity) {
        return wait_fast(bar, parity, abort_flag, status);
      };
      bool ok = true;
      while (ok) {
        if (!wait1(d_full(dq.slot), dq.phase)) break;
        const int nt = pieces[dq.slot].nt;
        const int halves = pieces[dq.slot].rows > 128 ? 2 : 1;
        mbar_arrive(d_empty(dq.slot));
        dq.next(kTcPieces);
        if (nt == 0) break;
        // step t: the products of tile t with V, and the scores of tile t + 1 (kApart: the scores
        // first, as soon as the half's of tile t have been read)
#pragma unroll 1
        for (int t = -1; ok && t < nt; ++t) {
          const bool more = t + 1 < nt;
          uint32_t ks = 0, vs = 0;
          auto queries = [&](int g) {
            if (!wait1(q_full(g), (pieces_of >> g) & 1u)) return false;
            pieces_of ^= 1u << g;
            tc_fence_after();
            return true;
          };
          auto scores = [&](int g, uint32_t col) {
            if (g == 0) {
              ks = rg.slot;
              if (!wait1(full(ks), rg.phase)) return false;
              rg.next(T::kStages);
            }
            const uint64_t qa = q_half + g * kStep, kb = k_ring + ks * kStep;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t at = (k / 4) * (kHalf >> 4) + (k % 4) * 2;
              mma_bf16(col, qa + at, kb + at, kIdS, k > 0);
            }
            mma_commit(s_full(g));
            if (g + 1 == halves) mma_commit(empty(ks));
            return true;
          };
          if (t >= 0) {
            vs = rg.slot;
            if (!(ok = wait1(full(vs), rg.phase))) break;
            rg.next(T::kStages);
          }
#pragma unroll 1
          for (int g = 0; g < halves; ++g) {
            const uint32_t col = tmem + (T::kApart ? 64u : 128u) * g;
            constexpr uint32_t kO = T::o_col(0), kP = T::p_col(0);
            if (T::kApart && more) {
              if (t < 0) {
                ok = queries(g);
              } else {
                ok = wait1(s_read(g), (tiles_of >> g) & 1u);
                tc_fence_after();
              }
              if (!(ok = ok && scores(g, tmem + T::s_col(g)))) break;
            }
            if (t >= 0) {
              // O += P V as the two 64-key halves of P arrive
              const uint64_t vb = v_ring + vs * kStep;
              const uint32_t par = (tiles_of >> g) & 1u;
              tiles_of ^= 1u << g;
              if (!(ok = wait1(p_full(g, 0), par))) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(col + kO, col + kP + 8u * k, vb + k * (2048 >> 4), kIdO, t > 0 || k > 0);
              mma_commit(pa_done(g));
              if (!(ok = wait1(p_full(g, 1), par))) break;
              tc_fence_after();
#pragma unroll
              for (int k = 4; k < 8; ++k)
                mma_ts(col + kO, col + kP + 8u * k, vb + k * (2048 >> 4), kIdO, 1u);
              mma_commit(pv_done(g));
              if (g + 1 == halves) mma_commit(empty(vs));
            } else if (!T::kApart && !(ok = queries(g))) {
              break;
            }
            if (!T::kApart && more && !(ok = scores(g, col))) break;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kTcCopyWarp || (!FP8 && warp == kTcCopyWarpV)) {
    // ------------------------------------------------------------ tile copies
    constexpr int kParts = FP8 ? 1 : D / 64;
    constexpr uint32_t kPitch = FP8 ? T::kRawPitch : 128;
    constexpr uint32_t kN = FP8 ? T::kRaw : T::kStages;
    const bool split = !FP8 && a.b.page_shift < kTcSplitShift;  // K and V by a warp each
    const bool take_k = warp == kTcCopyWarp, take_v = split ? !take_k : take_k;
    const int ps = 1 << a.b.page_shift;
    const int box_rows = min(ps, kAttnTK);
    const int boxes = kAttnTK / box_rows * kParts;  // <= 32: pages of at least 8 rows
    const int pl = lane / kParts, part = lane % kParts;
    const uint32_t box_bytes = (uint32_t)box_rows * kPitch;
    static_assert(FP8 || kN % 2 == 0, "K in the even stages, V in the odd ones");
    Ring rg{take_k ? 0u : 1u, 0};
    uint32_t issued = 0;
    auto fullb = [&](uint32_t s) { return FP8 ? raw_full(s) : full(s); };
    auto emptyb = [&](uint32_t s) { return FP8 ? raw_empty(s) : empty(s); };
    AttnRec* rec = &attn_scratch(a.scratch, kTcBR).rec[blockIdx.x];
    if (take_k && lane == 0) rec->starts = rec->mid = rec->ends = 0;
    auto drain_pieces = [&]() {  // a warp without work keeps the schedule going
      TcPiece p;
      while (get_piece(p)) {
      }
      return false;
    };
    TcPiece d, d2;  // the piece being copied, and the one after it
    // Publishes the next piece (nt = 0: none is left) and sends its query rows to L2: one run of
    // the group's heads per token.
    auto publish = [&](TcPiece& d) {
      AttnPiece p;
      const bool have = next_piece(a.b, sh, cur, p);
      d.nt = d.j0 = d.lo = d.hi = d.in_lo = d.in_hi = d.rows = d.r0 = 0;
      d.q0 = d.n = d.L = d.head = d.slot = d.seq = 0;
      if (have) {
        const KeyRange k0 = key_range(p.q, p.u.i0, sh.causal, sh.window);
        const KeyRange k1 = key_range(p.q, p.u.i1, sh.causal, sh.window);
        d.seq = p.s;
        d.nt = p.tb - p.ta;
        d.j0 = (p.u.t0 + p.ta) * kAttnTK;
        d.lo = p.u.lo;
        d.hi = p.u.hi;
        d.in_lo = max(k0.lo, k1.lo);
        d.in_hi = min(k0.hi, k1.hi);
        d.r0 = p.rb * kTcBR;
        d.rows = min(kTcBR, p.q.n * sh.G - d.r0);
        d.q0 = p.q.q0;
        d.n = p.q.n;
        d.L = p.q.L;
        d.head = p.head;
        d.slot = p.whole() ? -1 : p.first() ? 2 * (int)blockIdx.x + 1 : 2 * (int)blockIdx.x;
      }
      if (!wait(d_empty(dq.slot), dq.phase ^ 1u)) return false;
      if (lane == 0) {
        int4* dst = reinterpret_cast<int4*>(pieces + dq.slot);
        dst[0] = make_int4(d.nt, d.j0, d.lo, d.hi);
        dst[1] = make_int4(d.in_lo, d.in_hi, d.rows, d.r0);
        dst[2] = make_int4(d.q0, d.n, d.L, d.head);
        dst[3] = make_int4(d.slot, d.seq, 0, 0);
        mbar_arrive(d_full(dq.slot));
      }
      __syncwarp();
      dq.next(kTcPieces);
      if (have) {
        if (lane == 0 && p.first() && !p.last()) {
          rec->q0 = p.q.q0;
          rec->n = p.q.n;
          rec->head = p.head;
          rec->rb = p.rb;
          rec->starts = 1;
        } else if (lane == 0 && !p.first()) {
          rec->mid = 1;
          rec->ends = p.last();
        }
#pragma unroll 1
        for (int i = p.u.i0 + lane; i <= p.u.i1; i += 32)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                           static_cast<const __nv_bfloat16*>(a.q) +
                           (size_t)(p.q.q0 + i) * a.q_stride + (size_t)p.head * sh.G * D),
                       "r"(sh.G * D * 2)
                       : "memory");
      }
      return true;
    };
    bool ok = take_k ? publish(d) : split && get_piece(d);
    if (!take_k && !split) ok = drain_pieces();
    while (ok && d.nt > 0) {
      auto live_at = [&](int t) {
        const int j = d.j0 + t * kAttnTK + pl * box_rows;
        return t < d.nt && lane < boxes && j < d.hi && j + box_rows > d.lo;
      };
      auto page_at = [&](int t) {
        return live_at(t) ? page_of(a.b, d.seq, d.j0 + t * kAttnTK + pl * box_rows) : 0;
      };
      auto copy = [&](int t, int page, bool v) {
        const bool live = live_at(t);
        const uint32_t bytes = box_bytes * __popc(__ballot_sync(0xffffffffu, live));
        const uint32_t slot = rg.slot;
        if (!wait(emptyb(slot), rg.phase ^ 1u)) return false;
        // a V tile with positions that no row attends passes through the cleaning warp
        const int j = d.j0 + t * kAttnTK;
        const uint32_t bar = !FP8 && v && edge(d, j) ? v_raw(slot) : fullb(slot);
        if (lane == 0) mbar_expect_tx(bar, bytes);
        __syncwarp();
        if (live)
          tma_load_4d((FP8 ? codes + slot * T::kRawTile : ring + slot * T::kTile) + part * kHalf +
                          pl * box_bytes,
                      v ? &maps.v : &maps.k, bar, part * 64, (j + pl * box_rows) & (ps - 1),
                      d.head, page);
        ++issued;
        rg.next(kN);
        if (split) rg.next(kN);  // the other warp's stage
        return true;
      };
      int page = page_at(0);
      for (int t = 0; ok && t < d.nt; ++t) {
        const int next = page_at(t + 1);
        ok = (!take_k || copy(t, page, false)) && (!take_v || copy(t, page, true));
        page = next;
        if (ok && take_k && t == 0) ok = publish(d2);  // one piece ahead, behind the first copies
      }
      if (take_k) d = d2;
      else ok = ok && get_piece(d);
    }
    if (*abort_flag && lane == 0)  // let what is in flight land before the CTA can exit
      for (uint32_t i = 0; i < (issued < kN ? issued : kN); ++i)
        land(fullb((rg.slot + kN - 1 - i) % kN), rg.slot > i ? rg.phase : rg.phase ^ 1u);
    __syncwarp();
  } else if (!FP8 && warp == kTcCvtWarp) {
    // ------------------------------------------------------------ V tiles at the edges
    // v of positions that no row attends becomes 0, whatever the page holds (0 * NaN = NaN).
    // Only a unit's first tile (window) and last tile (length) have such positions.
    uint32_t at = 0, phases = 0;  // ring position of the piece, phase of each stage's v_raw
    bool ok = true;
    TcPiece p;
    while (ok && get_piece(p)) {
      for (int t = 0; ok && t < p.nt; t += max(1, p.nt - 1)) {
        const int j0 = p.j0 + t * kAttnTK;
        if (!edge(p, j0)) continue;
        const uint32_t slot = (at + 2 * t + 1) % T::kStages;
        if (!(ok = wait(v_raw(slot), (phases >> slot) & 1u))) break;
        phases ^= 1u << slot;
        const int lo = max(p.lo - j0, 0), hi = min(p.hi - j0, kAttnTK);
        for (int i = lane; i < kAttnTK * (D / 8); i += 32) {
          const int r = i / (D / 8), c = i % (D / 8);
          if (r < lo || r >= hi)
            sts128(ring + slot * T::kTile + (c / 8) * kHalf + r * 128 + (c & 7) * 16,
                   make_uint4(0u, 0u, 0u, 0u));
        }
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(slot));
      }
      at += 2 * p.nt;
    }
  } else if (FP8) {
    // ------------------------------------------------------------ codes to f16
    const int row0 = threadIdx.x - 32 * kTcCvtWarp;
    Ring rq{0, 0}, rg{0, 0};
    bool ok = true;
    auto convert = [&](const TcPiece& p, int t, bool v) {
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
        const int j = p.j0 + t * kAttnTK + row;
        if (v && (j < p.lo || j >= p.hi)) {  // no row attends it: 0, whatever the page holds
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
    TcPiece p;
    while (ok && get_piece(p)) {
      for (int t = 0; ok && t < p.nt; ++t) ok = convert(p, t, false) && convert(p, t, true);
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
  const auto sh = attn_shape<typename T::Shape>(a, 8, unit_cost(8, D, FP8, false));
  static_assert(kTcBR == 1 << 8, "rows per unit");
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
