// Rotary embedding of a batch's new tokens and the write of their k and v into the paged cache.
//
// The token at index i of its sequence sits at position p = kv_len - n + i; its k and v go to
// row p % page_size of page block_table[seq][p / page_size]. The first R columns of each q and
// k head turn by the angle of p, pair by pair, (a, b) -> (a cos - b sin, b cos + a sin), in
// fp32 from an fp32 table; q is rounded once to bf16, k and v once to the cache's type (e4m3:
// of x / scale, saturating at 448).
//
// One CTA per token; a thread handles two vectors of eight columns at a time,
// the two halves of eight pairs (half-split pairs) or sixteen neighbouring columns, and loads the
// next two before it stores these; the first are loaded before the token's sequence and page are
// known. 5,867 tokens of 32 + 2 x 8 heads of 128 into an e4m3 cache (134 MB) take 27.4 us, 4.9
// TB/s, and 27.4 into a bf16 cache (146 MB); 32 tokens 3.5 (4.1 when the lookups come first). HBM
// would need 20 of the 27.4 us, and with half of the writes still in L2 it carries 3.3 TB/s at 49 %
// of the warps active: a CTA's loads of bounds, length, page and angles follow one another, before
// two rounds of work, in six to seven waves of CTAs. Six CTAs of 192 threads on an SM: with
// eight the registers spill (34 us), three of 384 take 33, and several tokens a CTA with their
// lookups side by side 46.
#include "block.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace gbmoe {
namespace {

constexpr int kAppendThreads = 192, kAppendCtas = 6;

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  u.x = pack_bf16x2(v[0], v[1]);
  u.y = pack_bf16x2(v[2], v[3]);
  u.z = pack_bf16x2(v[4], v[5]);
  u.w = pack_bf16x2(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&v)[8], float s, float inv) {
  uint2 c;
  c.x = e4m3x4_divided<true>(v[0], v[1], v[2], v[3], s, inv);
  c.y = e4m3x4_divided<true>(v[4], v[5], v[6], v[7], s, inv);
  *reinterpret_cast<uint2*>(p) = c;
}
__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Two vectors of eight columns of one head of a token: columns c0 and c1 of q (kind 0), k or v.
struct Item {
  int kind, h, p, c0, c1;
  bool turn;
  uint4 a, b;  // as loaded
};
__device__ __forceinline__ Item load_item(const KvAppendArgs& a, int t, int it) {
  Item x;
  const int per_head = a.D / 16;
  x.h = it / per_head;
  x.p = it % per_head;
  x.kind = x.h < a.hq ? 0 : (x.h < a.hq + a.hkv ? 1 : 2);
  x.h -= x.kind == 0 ? 0 : (x.kind == 1 ? a.hq : a.hq + a.hkv);
  x.turn = x.kind < 2 && x.p < a.rotary / 16;
  const bool split = x.turn && !a.interleaved;
  x.c0 = split ? 8 * x.p : 16 * x.p;
  x.c1 = split ? 8 * x.p + a.rotary / 2 : 16 * x.p + 8;
  const __nv_bfloat16* src =
      x.kind == 0 ? static_cast<const __nv_bfloat16*>(a.q) + (size_t)t * a.q_stride
      : x.kind == 1 ? static_cast<const __nv_bfloat16*>(a.k) + (size_t)t * a.k_stride
                    : static_cast<const __nv_bfloat16*>(a.v) + (size_t)t * a.v_stride;
  src += (size_t)x.h * a.D;
  x.a = __ldg(reinterpret_cast<const uint4*>(src + x.c0));
  x.b = __ldg(reinterpret_cast<const uint4*>(src + x.c1));
  return x;
}

template <bool FP8>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas) kv_append_kernel(KvAppendArgs a) {
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int items = (a.hq + 2 * a.hkv) * (a.D / 16);
  Item next;  // the first vectors are under way while the token's place is looked up
  if ((int)threadIdx.x < items) next = load_item(a, t, threadIdx.x);
  const int s = find_seq_warp(a.b, t, lane);  // every warp finds it: no barrier
  if (s < 0) return;                          // a token of no sequence (padding)
  const SeqInfo q = seq_info(a.b, s);
  const int pos = q.L - q.n + (t - q.q0);
  if (t - q.q0 >= q.n || pos < 0 || (a.cos_sin && pos >= a.max_pos)) {
    if (threadIdx.x == 0) record_status(a.b.status, GBMOE_ERR_DEVICE_CHECK);
    return;
  }
  bool bad = false;
  const int page =
      checked_page(__ldg(a.b.table + (size_t)s * a.b.table_stride + (pos >> a.b.page_shift)),
                   a.b.num_pages, &bad);
  if (bad && threadIdx.x == 0) record_status(a.b.status, GBMOE_ERR_DEVICE_CHECK);
  const size_t row = (size_t)page * a.c.page_stride +
                     (size_t)(pos & ((1 << a.b.page_shift) - 1)) * a.c.token_stride;
  const int R = a.rotary;
  const float* cs = a.cos_sin ? a.cos_sin + (size_t)pos * R : nullptr;
  for (int it = threadIdx.x; it < items; it += blockDim.x) {
    const Item now = next;
    if (it + (int)blockDim.x < items) next = load_item(a, t, it + blockDim.x);
    const int kind = now.kind, h = now.h, p = now.p, c0 = now.c0, c1 = now.c1;
    const bool turn = now.turn, split = turn && !a.interleaved;
    float x[8], y[8];
    unpack8(now.a, x);
    unpack8(now.b, y);
    if (turn) {
      float c[8], z[8];
      load8f(cs + 8 * p, c);
      load8f(cs + R / 2 + 8 * p, z);
      if (split) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = x[i] * c[i] - y[i] * z[i];
          y[i] = y[i] * c[i] + x[i] * z[i];
          x[i] = u;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = x[2 * i] * c[i] - x[2 * i + 1] * z[i];
          x[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * z[i];
          x[2 * i] = u;
          const float w = y[2 * i] * c[4 + i] - y[2 * i + 1] * z[4 + i];
          y[2 * i + 1] = y[2 * i + 1] * c[4 + i] + y[2 * i] * z[4 + i];
          y[2 * i] = w;
        }
      }
    }
    if (kind == 0) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.q_out) + ((size_t)t * a.hq + h) * a.D;
      store8(dst + c0, x);
      store8(dst + c1, y);
    } else if (!bad) {
      const size_t at = row + (size_t)h * a.c.head_stride;
      if (FP8) {
        uint8_t* dst = static_cast<uint8_t*>(kind == 1 ? a.c.k : a.c.v) + at;
        const float s = kind == 1 ? a.k_scale : a.v_scale, inv = kind == 1 ? a.k_inv : a.v_inv;
        store8_e4m3(dst + c0, x, s, inv);
        store8_e4m3(dst + c1, y, s, inv);
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(kind == 1 ? a.c.k : a.c.v) + at;
        store8(dst + c0, x);
        store8(dst + c1, y);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  if (a.fp8)
    launch_kernel(kv_append_kernel<true>, dim3(a.b.T), dim3(kAppendThreads), 0, stream, a);
  else
    launch_kernel(kv_append_kernel<false>, dim3(a.b.T), dim3(kAppendThreads), 0, stream, a);
  return cudaGetLastError();
}

}  // namespace gbmoe
