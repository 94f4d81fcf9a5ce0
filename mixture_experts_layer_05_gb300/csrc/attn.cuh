// Device side of paged attention's work split (attn_plan.h), shared by the two attention kernels:
// every CTA finds its range of the line of tiles, walks its pieces, and leaves the pieces of cut
// units in the workspace. attn_decode.cu joins those itself; after attn_tc.cu's kernel, which
// also leaves a record per CTA, attn_join_kernel does.
#pragma once

#include "attn_plan.h"
#include "block.cuh"
#include "tc.cuh"

namespace gbmoe {

constexpr int kAttnMaxBR = 256;    // rows per unit of the widest kernel

// What a CTA's cut units look like, for attn_join_kernel: the unit that it begins and leaves
// to the next CTA (starts), whether its first piece is of a unit begun before it (mid), and
// whether that unit ends there.
struct AttnRec {
  int starts, rb;
  int mid, ends;
  int q0, n, head, pad;  // the begun unit's sequence and kv head
};

// The workspace after the status region: records, then per CTA two piece slots (2c: a unit begun
// by an earlier CTA; 2c + 1: a unit left to the next) of (m, l) pairs and fp32 output rows.
struct AttnScratch {
  AttnRec* rec;
  float2* ml;   // [slot][BR]
  float* o;     // [slot][BR][D]
};
__host__ __device__ inline AttnScratch attn_scratch(void* base, int BR) {
  AttnScratch s;
  char* p = static_cast<char*>(base);
  s.rec = reinterpret_cast<AttnRec*>(p);
  p += kAttnMaxCtas * sizeof(AttnRec);
  s.ml = reinterpret_cast<float2*>(p);
  p += (size_t)kAttnMaxCtas * 2 * BR * sizeof(float2);
  s.o = reinterpret_cast<float*>(p);
  return s;
}

namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The line, the CTAs that share it, and the end of this one's range.
struct AttnSpan {
  int W, end, ctas;
};
// The CTA whose range holds the place x of the line.
__device__ __forceinline__ int cta_of(const AttnSpan& s, int x) {
  int c = (int)((float)x * s.ctas / s.W);
  c = min(max(c, 0), s.ctas - 1);
  while (range_at(s.W, c + 1, s.ctas) <= x) ++c;
  while (range_at(s.W, c, s.ctas) > x) --c;
  return c;
}

// The cursor with the sizes of its sequence qs at hand: reading them again costs a trip to L2 each
// time a piece is worked out, and the first piece waits for that.
struct AttnWalk : AttnCursor {
  int qs;
  SeqInfo q;
};

constexpr int kPlanBlocks = 4;  // row blocks that one thread adds up by itself

// The cursor `rem` into sequence s of sizes q, whose length on the line is `len`; a range of `left`
// lies ahead. Whole warps call it.
template <class Shape>
__device__ __forceinline__ void enter(const Shape& sh, const SeqInfo& q, int s, int rem,
                                      int len, int left, AttnWalk& c) {
  const int lane = threadIdx.x & 31;
  const int head = len / sh.hkv;  // length of one head
  c.s = c.qs = s;
  c.q = q;
  c.left = left;
  c.head = rem / head;
  rem -= c.head * head;
  const int blocks = unit_blocks(sh, q.n);
  if (blocks <= kPlanBlocks) {
    walk_blocks(sh, q, rem, c);
    return;
  }
  // the row block, 32 at a time
#pragma unroll 1
  for (; c.rb < blocks; c.rb += 32) {
    const int rb = c.rb + lane;
    int at = rb < blocks ? unit_length(sh, q, rb) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += v;
    }
    const uint32_t behind = __ballot_sync(0xffffffffu, at <= rem);
    if (behind != 0xffffffffu) {
      const int k = __popc(behind);  // whole units behind the cursor
      if (k > 0) rem -= __shfl_sync(0xffffffffu, at, k - 1);
      c.rb += k;
      break;
    }
    rem -= __shfl_sync(0xffffffffu, at, 31);
  }
  c.off = rem;
}

// This CTA's cursor; every thread of the block calls it. line: shared memory for S + 1 prefix
// sums, wsum: 32 more. A thread takes a sequence of few row blocks (single tokens), a warp one of
// many: a prompt of 8191 tokens has 128, and one thread walking them cost 45 us.
template <class Shape>
__device__ __forceinline__ AttnWalk attn_plan(const PagedBatch& b, const Shape& sh,
                                              int* line, int* wsum, AttnSpan& span) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int warps = nt >> 5;
  bool falls = false;
#pragma unroll 1
  for (int s = tid; s < b.S; s += nt) {
    const SeqInfo q = seq_info(b, s);
    falls |= b.cu[s + 1] < b.cu[s];
    line[s + 1] = unit_blocks(sh, q.n) <= kPlanBlocks ? seq_length(sh, q) * sh.hkv : -1;
  }
  if (tid == 0) line[0] = 0;
  falls = __syncthreads_or(falls);
  // few sequences: every warp looks through all and takes each `warps`-th; many: 32 apiece
  const bool few = b.S <= 1024;
  int mine = 0;
#pragma unroll 1
  for (int s0 = few ? 0 : warp * 32; s0 < b.S; s0 += few ? 32 : warps * 32) {
    uint32_t many = __ballot_sync(0xffffffffu, s0 + lane < b.S && line[s0 + lane + 1] < 0);
#pragma unroll 1
    while (many) {
      const int s = s0 + __ffs(many) - 1;
      many &= many - 1;
      if (few && mine++ % warps != warp) continue;
      const SeqInfo q = seq_info(b, s);
      const int blocks = unit_blocks(sh, q.n);
      int t = 0;
#pragma unroll 1
      for (int rb = lane; rb < blocks; rb += 32) t += unit_length(sh, q, rb);
      t = __reduce_add_sync(0xffffffffu, t);
      if (lane == 0) line[s + 1] = -2 - t * sh.hkv;  // marked until every warp has looked
    }
  }
  __syncthreads();
  AttnWalk c;
  c.s = c.head = c.rb = c.off = c.left = 0;
  c.qs = -1;
  span.W = span.ctas = span.end = 0;
  if (falls) {
    // Bounds that go back (reported already) let sequences share tokens: the length of the line is
    // then not bounded by the batch's, and one that leaves 32 bits gets no work at all.
    long long all = 0;
#pragma unroll 1
    for (int s = 0; s < b.S; ++s) all += line[s + 1] < 0 ? -2 - line[s + 1] : line[s + 1];
    if (all > 0x7fffffff) return c;
    __syncthreads();
  }
  // prefix sums: a run of sequences per thread
  const int per = (b.S + nt - 1) / nt;
  const int s0 = min(tid * per, b.S), s1 = min(s0 + per, b.S);
  int sum = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const int v = line[s + 1];
    sum += v < 0 ? -2 - v : v;
    line[s + 1] = sum;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int base = inc - sum;
#pragma unroll 1
  for (int w = 0; w < warp; ++w) base += wsum[w];
#pragma unroll 1
  for (int s = s0; s < s1; ++s) line[s + 1] += base;
  __syncthreads();
  const int W = line[b.S];
  span.W = W;
  span.ctas = line_ctas(sh, W, gridDim.x);  // every one of these has some of the line
  if ((int)blockIdx.x < span.ctas) {
    const int a = range_at(W, blockIdx.x, span.ctas);
    span.end = range_at(W, blockIdx.x + 1, span.ctas);
    int lo = 0, hi = b.S;  // the sequence with line[s] <= a < line[s + 1]
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (line[mid] <= a) lo = mid;
      else hi = mid;
    }
    enter(sh, seq_info(b, lo), lo, a - line[lo], line[lo + 1] - line[lo], span.end - a, c);
  }
  return c;
}

// The same by a warp alone, for few sequences (quick_plan): a lane holds a sequence, nothing
// goes through shared memory, and the warps that need no cursor go on. One small step takes 10.1
// us (10.9 when the whole block plans), packed prompts 85.2 (88.5).
__device__ __forceinline__ bool quick_plan(const PagedBatch& b, const AttnShape& sh) {
  return b.S <= 32 && (long long)b.T * sh.G <= 1024ll << sh.br_shift;
}
template <class Shape>
__device__ __forceinline__ AttnWalk attn_plan_warp(const PagedBatch& b, const Shape& sh,
                                                   AttnSpan& span) {
  const int lane = threadIdx.x & 31;
  AttnWalk c;
  c.s = c.head = c.rb = c.off = c.left = 0;
  c.qs = -1;
  span.W = span.ctas = span.end = 0;
  SeqInfo q{0, 0, 0};
  bool falls = false;
  int v = 0;
  if (lane < b.S) {
    q = seq_info(b, lane);
    falls = b.cu[lane + 1] < b.cu[lane];
    if (unit_blocks(sh, q.n) <= kPlanBlocks) v = seq_length(sh, q) * sh.hkv;
  }
  uint32_t many = __ballot_sync(0xffffffffu, unit_blocks(sh, q.n) > kPlanBlocks);
#pragma unroll 1
  while (many) {
    const int s = __ffs(many) - 1;
    many &= many - 1;
    const SeqInfo x{__shfl_sync(0xffffffffu, q.q0, s), __shfl_sync(0xffffffffu, q.n, s),
                    __shfl_sync(0xffffffffu, q.L, s)};
    const int blocks = unit_blocks(sh, x.n);
    int t = 0;
#pragma unroll 1
    for (int rb = lane; rb < blocks; rb += 32) t += unit_length(sh, x, rb);
    t = __reduce_add_sync(0xffffffffu, t);
    if (lane == s) v = t * sh.hkv;
  }
  if (__any_sync(0xffffffffu, falls)) {  // as above
    float all = (float)v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (all > 2147480000.f) return c;
  }
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  const int W = __shfl_sync(0xffffffffu, inc, 31);
  span.W = W;
  span.ctas = line_ctas(sh, W, gridDim.x);
  if ((int)blockIdx.x < span.ctas) {
    const int a = range_at(W, blockIdx.x, span.ctas);
    span.end = range_at(W, blockIdx.x + 1, span.ctas);
    const int lo = __popc(__ballot_sync(0xffffffffu, inc <= a));
    const SeqInfo x{__shfl_sync(0xffffffffu, q.q0, lo), __shfl_sync(0xffffffffu, q.n, lo),
                    __shfl_sync(0xffffffffu, q.L, lo)};
    enter(sh, x, lo, a - __shfl_sync(0xffffffffu, inc - v, lo), __shfl_sync(0xffffffffu, v, lo),
          span.end - a, c);
  }
  return c;
}

// The next piece of the cursor's range, false when none is left; sequences without rows and
// units of which the range holds only the extra cost are passed over.
template <class Shape>
__device__ __forceinline__ bool next_piece(const PagedBatch& b, const Shape& sh,
                                           AttnWalk& c, AttnPiece& p) {
#pragma unroll 1
  while (c.left > 0) {
#pragma unroll 1
    while (c.qs != c.s) {
      c.qs = c.s;
      c.q = seq_info(b, c.s);
      if (c.q.n == 0 && c.s + 1 < b.S) ++c.s;
    }
    p = take_piece(sh, c.q, c);
    if (p.ta < p.tb) return true;
  }
  return false;
}

// 4-D tile load (column, row of the page, head, page).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Box of a cache tile: up to 128 columns' bytes x box rows of one page and head.
bool make_cache_map(CUtensorMap* m, const void* ptr, const AttnArgs& a) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const int es = a.fp8 ? 1 : 2;
  const uint64_t ps = 1ull << a.b.page_shift;
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, ps, (cuuint64_t)a.hkv, (cuuint64_t)a.b.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)a.c.token_stride * es,
                                 (cuuint64_t)a.c.head_stride * es,
                                 (cuuint64_t)a.c.page_stride * es};
  const cuuint32_t inner = a.D * es < 128 ? a.D : 128 / es;
  const cuuint32_t box[4] = {inner, (cuuint32_t)(ps < kAttnTK ? ps : kAttnTK), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  // L2 fetches no more than a row of the head holds: what follows it belongs to other heads,
  // whose CTAs are elsewhere in the sequence
  const int run = a.c.token_stride == a.D ? 256 : a.D * es;
  const CUtensorMapL2promotion fetch = run >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                       : run >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                    : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  return enc(m, a.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             inner * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Joins the pieces of the units that CTA boundaries cut. Block (c, y): rows [32 y, 32 y + 32) of
// the unit that CTA c began and did not finish: sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i
// over its pieces in order, M = max m_i: 8 threads a row, four columns each in turn.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a, AttnShape sh, int ctas) {
  constexpr int C = D / 32;  // vectors of four columns per thread
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const AttnScratch sc = attn_scratch(a.scratch, 1 << sh.br_shift);
  const int c0 = blockIdx.x;
  const int row = blockIdx.y * 32 + threadIdx.x / 8, col = threadIdx.x % 8 * 4;
  // everything that does not wait for something else is loaded at once: the record, the records
  // of the CTAs after c0, and the first two pieces (most units have no more)
  const AttnRec rec = sc.rec[c0];
  int2 held[kAttnMaxCtas / 32];  // (mid, ends)
#pragma unroll
  for (int i = 0; i < kAttnMaxCtas / 32; ++i) {
    const int c = c0 + 1 + 32 * i + lane;
    held[i] = c < ctas ? *reinterpret_cast<const int2*>(&sc.rec[c].mid) : make_int2(0, 0);
  }
  const size_t first = ((size_t)(2 * c0 + 1) << sh.br_shift) + row;
  float2 ml = sc.ml[first];
  float4 o[C];
#pragma unroll
  for (int i = 0; i < C; ++i)
    o[i] = *reinterpret_cast<const float4*>(sc.o + first * D + col + 32 * i);
  if (!rec.starts) return;
  int c1 = ctas - 1;
#pragma unroll
  for (int i = kAttnMaxCtas / 32 - 1; i >= 0; --i) {
    const uint32_t end = __ballot_sync(0xffffffffu, held[i].x && held[i].y);
    if (end) c1 = c0 + 32 * i + __ffs(end);
  }
  const int ur = (rec.rb << sh.br_shift) + row;
  const bool valid = ur < rec.n * sh.G;
  float M = ml.x, l = ml.y;
#pragma unroll 2
  for (int c = c0 + 1; c <= c1; ++c) {
    if (!sc.rec[c].mid) continue;
    const size_t at = ((size_t)(2 * c) << sh.br_shift) + row;
    const float2 next = sc.ml[at];
    float4 v[C];
#pragma unroll
    for (int i = 0; i < C; ++i)
      v[i] = *reinterpret_cast<const float4*>(sc.o + at * D + col + 32 * i);
    const float Mn = fmaxf(M, next.x), Ms = Mn == -INFINITY ? 0.f : Mn;
    const float f = ex2(M - Ms), w = ex2(next.x - Ms);
    M = Mn;
    l = l * f + next.y * w;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      o[i].x = o[i].x * f + v[i].x * w;
      o[i].y = o[i].y * f + v[i].y * w;
      o[i].z = o[i].z * f + v[i].z * w;
      o[i].w = o[i].w * f + v[i].w * w;
    }
  }
  if (!valid) return;
  const size_t orow = (size_t)(rec.q0 + div_group(sh, ur)) * a.hq + rec.head * sh.G +
                      (ur - div_group(sh, ur) * sh.G);
  const float inv = l == 0.f ? 0.f : a.v_scale / l;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    uint2 w;
    w.x = pack_bf16x2(o[i].x * inv, o[i].y * inv);
    w.y = pack_bf16x2(o[i].z * inv, o[i].w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + col + 32 * i) = w;
  }
  if (a.lse && col == 0)
    a.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

// Shape of a launch whose units have 1 << br_shift rows.
template <class Shape = AttnShape>
Shape attn_shape(const AttnArgs& a, int br_shift, int extra) {
  Shape sh;
  set_group(sh, a.hq / a.hkv);
  sh.hkv = a.hkv;
  sh.br_shift = br_shift;
  sh.extra = extra;
  sh.causal = a.causal;
  sh.window = a.window;
  return sh;
}

cudaError_t launch_attn_join(const AttnArgs& a, const AttnShape& sh, int ctas,
                             cudaStream_t stream) {
  const dim3 grid(ctas, (1 << sh.br_shift) / 32);
  if (a.D == 64) launch_kernel(attn_join_kernel<64>, grid, dim3(256), 0, stream, a, sh, ctas);
  else launch_kernel(attn_join_kernel<128>, grid, dim3(256), 0, stream, a, sh, ctas);
  return cudaGetLastError();
}

}  // namespace
}  // namespace gbmoe
