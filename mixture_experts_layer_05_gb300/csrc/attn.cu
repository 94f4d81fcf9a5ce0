// Attention of each sequence's new tokens over its paged cache: one warp per (token, query
// head), one pass over the keys with the running maximum and sum of the softmax.
#include <cuda_fp8.h>

#include "block.cuh"
#include "kernels.h"

namespace gbmoe {
namespace {

template <bool FP8, int PER>
__device__ __forceinline__ void load_row(const void* base, size_t at, int lane, float (&v)[PER]) {
  if (FP8) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + at + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      __nv_fp8_e4m3 c;
      c.__x = p[i];
      v[i] = (float)c;
    }
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + at + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = __bfloat162float(p[i]);
  }
}

template <bool FP8, int D>
__global__ void __launch_bounds__(256) attn_row_kernel(AttnArgs a) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= (long long)a.b.T * a.hq) return;
  const int t = (int)(w / a.hq), h = (int)(w % a.hq);
  const int s = find_seq_warp(a.b, t, lane);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (size_t)w * D + lane * PER;
  float o[PER], q[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  if (s >= 0) {
    const SeqInfo sq = seq_info(a.b, s);
    if (t - sq.q0 < sq.n) {
      const KeyRange r = key_range(sq, t - sq.q0, a.causal, a.window);
      load_row<false, PER>(a.q, (size_t)t * a.q_stride + (size_t)h * D, lane, q);
      const size_t head = (size_t)(h / (a.hq / a.hkv)) * a.c.head_stride;
      for (int j = r.lo; j < r.hi; ++j) {
        const int page = page_of(a.b, s, j);
        const size_t at = (size_t)page * a.c.page_stride +
                          (size_t)(j & ((1 << a.b.page_shift) - 1)) * a.c.token_stride + head;
        float k[PER], v[PER];
        load_row<FP8, PER>(a.c.k, at, lane, k);
        load_row<FP8, PER>(a.c.v, at, lane, v);
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) d = fmaf(q[i], k[i], d);
        d = warp_sum(d) * a.scale_log2;
        const float mn = fmaxf(m, d);
        const float c = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float p = mn == -INFINITY ? 0.f : exp2f(d - mn);
        l = l * c + p;
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = fmaf(p, v[i], o[i] * c);
        m = mn;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : a.v_scale / l;  // no key: zeros
#pragma unroll
  for (int i = 0; i < PER; ++i) out[i] = __float2bfloat16(o[i] * inv);
  if (a.lse && lane == 0)
    a.lse[w] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
}

}  // namespace

size_t attn_scratch_bytes(int) { return 0; }

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  const long long warps = (long long)a.b.T * a.hq;
  const dim3 grid((unsigned)((warps + 7) / 8));
  if (a.fp8) {
    if (a.D == 64) launch_kernel(attn_row_kernel<true, 64>, grid, dim3(256), 0, stream, a);
    else launch_kernel(attn_row_kernel<true, 128>, grid, dim3(256), 0, stream, a);
  } else {
    if (a.D == 64) launch_kernel(attn_row_kernel<false, 64>, grid, dim3(256), 0, stream, a);
    else launch_kernel(attn_row_kernel<false, 128>, grid, dim3(256), 0, stream, a);
  }
  return cudaGetLastError();
}

}  // namespace gbmoe
