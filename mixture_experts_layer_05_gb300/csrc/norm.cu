// RMS norm with the residual's addition and an optional 8-bit output:
//
//   h = x + residual            residual_out = bf16(h)
//   y = h * rsqrt(mean(h^2) + eps) * w
//   s = max(max |y over 128 columns|, 1e-10) / 448,  q = e4m3(y / s)
//
// All sums and y are fp32; y is rounded once, to bf16 or (from fp32, not from the bf16 y) to
// e4m3. One CTA per row: the row stays in registers between the sum of squares and the
// outputs, so each input is read once. Thread i holds the vectors of eight columns i, i +
// blockDim, ..., so 16 neighbouring threads hold one 128-column group and find its largest
// magnitude with four shuffles.
#include "block.h"
#include "fp8.cuh"
#include "kernels.h"

namespace gbmoe {
namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxVec = 4;  // vectors of eight columns per thread

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
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

template <int VEC>
__global__ void __launch_bounds__(kNormMaxThreads) rms_norm_kernel(RmsNormArgs a) {
  __shared__ float red[32];
  const int t = blockIdx.x;
  const int nv = a.H / 8;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + (size_t)t * a.x_stride;
  const __nv_bfloat16* r =
      a.residual ? static_cast<const __nv_bfloat16*>(a.residual) + (size_t)t * a.residual_stride
                 : nullptr;
  const __nv_bfloat16* wt = static_cast<const __nv_bfloat16*>(a.weight);
  float h[VEC][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
    if (v < nv) {
      load8(x + v * 8, h[i]);
      if (r) {
        float u[8];
        load8(r + v * 8, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += u[j];
        if (a.residual_out)
          store8(static_cast<__nv_bfloat16*>(a.residual_out) + (size_t)t * a.H + v * 8, h[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
  }
  ss = warp_sum(ss);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  ss = warp_sum((int)(threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f);
  const float rs = 1.f / sqrtf(ss / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float y[8], amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = 0.f;
    if (v < nv) {
      float w[8];
      load8(wt + v * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = h[i][j] * rs * w[j];
        amax = fmaxf(amax, fabsf(y[j]));
      }
      if (a.y) store8(static_cast<__nv_bfloat16*>(a.y) + (size_t)t * a.H + v * 8, y);
    }
    if (a.q) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (v < nv) {
        const float s = fp8_group_scale(amax);
        uint2 c;
        c.x = e4m3x4(y[0], y[1], y[2], y[3], s);
        c.y = e4m3x4(y[4], y[5], y[6], y[7], s);
        *reinterpret_cast<uint2*>(a.q + (size_t)t * a.H + v * 8) = c;
        if ((threadIdx.x & 15) == 0) a.scale[(size_t)(v / 16) * a.T + t] = s;
      }
    }
  }
}

}  // namespace

int rms_norm_max_hidden() { return kNormMaxThreads * kNormMaxVec * 8; }

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t stream) {
  const int nv = a.H / 8;
  const int vec = (nv + kNormMaxThreads - 1) / kNormMaxThreads;
  int threads = (nv + vec - 1) / vec;
  threads = (threads + 31) / 32 * 32;
  auto go = [&](auto k) { launch_kernel(k, dim3(a.T), dim3(threads), 0, stream, a); };
  if (vec == 1) go(rms_norm_kernel<1>);
  else if (vec == 2) go(rms_norm_kernel<2>);
  else go(rms_norm_kernel<4>);
  return cudaGetLastError();
}

}  // namespace gbmoe
