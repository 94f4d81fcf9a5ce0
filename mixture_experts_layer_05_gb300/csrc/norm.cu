// RMS norm with the residual's addition and an optional 8-bit output:
//
//   h = x + residual            residual_out = bf16(h)
//   y = h * rsqrt(mean(h^2) + eps) * w
//   s = max(max |y over 128 columns|, 1e-10) / 448,  q = e4m3(y / s)
//
// All sums and y are fp32; y is rounded once, to bf16 or (from fp32, not from the bf16 y) to
// e4m3. A row stays in registers between the sum of squares and the outputs, so each input is
// read once. Thread i holds the vectors of eight columns i, i + blockDim, ..., so 16
// neighbouring threads hold one 128-column group and find its largest magnitude with four
// shuffles.
//
// Bound by HBM. A CTA per row. Up to two rows an SM a thread holds one vector, the shortest
// chain; beyond that two (half the threads per row, so that more rows are in different phases on
// an SM). 8192 x 7168 with a residual and both outputs, 530 MB: 79 us (6.7 TB/s, the rate of a
// plain copy); 88 with one vector per thread, 81 with four, 126 with CTAs that stay and bulk
// copies of the next rows into shared memory. A division of each value by its group's
// scale cost 30 us of arithmetic; a product with the reciprocal and its correction cost none.
#include "block.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace gbmoe {
namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxVec = 4;  // vectors of eight columns per thread

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

// One row's outputs from its h (fp32, this thread's vectors) and the sum of squares.
template <int VEC>
__device__ __forceinline__ void write_row(const RmsNormArgs& a, int t, int nv, float ss,
                                          const float (&h)[VEC][8]) {
  // the root is corrected once by what it leaves (Newton's step); rounded forms of the mean's
  // division and the root need more registers and cost 7 us of 62 in 8192 rows
  const float var = fmaf(ss, a.inv_h, a.eps), r0 = rsqrtf(var), left = fmaf(-var * r0, r0, 1.f);
  const float rs = left == left ? fmaf(0.5f * r0, left, r0) : r0;  // NaN: var is 0 or infinite
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float y[8], amax = 0.f;
    unpack8(v < nv ? __ldg(static_cast<const uint4*>(a.weight) + v) : make_uint4(0u, 0u, 0u, 0u), y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = y[j] * h[i][j] * rs;  // the first product is exact without a residual
      amax = fmaxf(amax, fabsf(y[j]));
    }
    if (a.y && v < nv) store8(static_cast<__nv_bfloat16*>(a.y) + (size_t)t * a.H + v * 8, y);
    if (a.q) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (v < nv) {
        const float s = fp8_group_scale(amax);
        uint2 c;
        // an infinite scale (1 / s = 0) leaves the products as they are
        const float inv = __fdiv_rn(1.f, s), back = s < INFINITY ? s : 0.f;
        c.x = e4m3x4_divided<false>(y[0], y[1], y[2], y[3], back, inv);
        c.y = e4m3x4_divided<false>(y[4], y[5], y[6], y[7], back, inv);
        *reinterpret_cast<uint2*>(a.q + (size_t)t * a.H + v * 8) = c;
        if ((threadIdx.x & 15) == 0) a.scale[(size_t)(v / 16) * a.T + t] = s;
      }
    }
  }
}

// h = x + r of one vector, and its squares added to ss.
__device__ __forceinline__ void add_vec(const uint4& x, const uint4& r, float (&h)[8], float& ss) {
  float u[8];
  unpack8(x, h);
  unpack8(r, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h[j] += u[j];
    ss = fmaf(h[j], h[j], ss);
  }
}

// A row per CTA. Up to two vectors a thread, 32 registers: at 37 the rows on an SM fall from four
// to three, and 8192 x 7168 without residual takes 46 us for 41.
template <int VEC>
__global__ void __launch_bounds__(kNormMaxThreads, VEC <= 2 ? 2 : 1)
    rms_norm_kernel(RmsNormArgs a) {
  __shared__ float red[32];
  const int nv = a.H / 8, t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) +
                                                  (size_t)t * a.x_stride);
  const uint4* r = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.residual) +
                                                  (size_t)t * a.residual_stride);
  uint4 xv[VEC], rv[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    xv[i] = rv[i] = zero;
    if (v < nv) {
      xv[i] = x[v];
      if (a.residual) rv[i] = r[v];
    }
  }
  float h[VEC][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    add_vec(xv[i], rv[i], h[i], ss);
    if (a.residual_out && v < nv)
      store8(static_cast<__nv_bfloat16*>(a.residual_out) + (size_t)t * a.H + v * 8, h[i]);
  }
  ss = warp_sum(ss);
  if (lane == 0) red[warp] = ss;
  __syncthreads();
  write_row(a, t, nv, warp_sum(lane < nw ? red[lane] : 0.f), h);
}

}  // namespace

int rms_norm_max_hidden() { return kNormMaxThreads * kNormMaxVec * 8; }

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t stream) {
  const int nv = a.H / 8;
  // up to two rows an SM: a vector per thread; more: two, when a row has that many
  const int wide = a.T <= 2 * num_sms() ? kNormMaxThreads : kNormMaxThreads / 2;
  int vec = (nv + wide - 1) / wide;
  if (vec > 2) vec = 4;
  const int threads = ((nv + vec - 1) / vec + 31) / 32 * 32;
  auto go = [&](auto k) { launch_kernel(k, dim3(a.T), dim3(threads), 0, stream, a); };
  if (vec == 1) go(rms_norm_kernel<1>);
  else if (vec == 2) go(rms_norm_kernel<2>);
  else go(rms_norm_kernel<4>);
  return cudaGetLastError();
}

}  // namespace gbmoe
