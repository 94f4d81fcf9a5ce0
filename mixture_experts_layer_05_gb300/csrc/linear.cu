// moe_linear and moe_grouped_linear: out = bf16(act(x w[g]^T + bias[g]) * row_weight + residual) over
// the rows of each group. A thread owns one output column of a block of 16 rows of one group.
#include <cuda_fp8.h>

#include "common.cuh"
#include "linear.h"

namespace gbmoe {
namespace {

constexpr int kRows = 16, kCols = 128, kStep = 128;

__device__ __forceinline__ float value(const void* p, long long i, bool fp8) {
  if (!fp8) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  __nv_fp8_e4m3 v;
  v.__x = static_cast<const uint8_t*>(p)[i];
  return (float)v;
}

__device__ float activated(float z, int act) {
  switch (act) {
    case GBMOE_EPI_RELU: return z < 0.f ? 0.f : z;
    case GBMOE_EPI_SILU: return z / (1.f + __expf(-z));
    case GBMOE_EPI_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678f));
    case GBMOE_EPI_GELU_TANH:
      return 0.5f * z * (1.f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}

// Sums of column n of group g over the block's rows [r0, r0 + rows).
__device__ void column(const LinearArgs& a, int g, int n, int r0, int rows, float (&acc)[kRows],
                       float (*xs)[kStep]) {
  const int kb_count = (a.K + kStep - 1) / kStep;
  for (int i = 0; i < kRows; ++i) acc[i] = 0.f;
  for (int kb = 0; kb < kb_count; ++kb) {
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kStep; i += blockDim.x) {
      const int r = i / kStep, k = kb * kStep + i % kStep;
      float v = 0.f;
      if (r < rows && k < a.K) {
        v = value(a.x, (long long)(r0 + r) * a.x_stride + k, a.fp8);
        if (a.fp8) v *= a.x_scale[(long long)kb * a.T + r0 + r];
      }
      xs[r][i % kStep] = v;
    }
    __syncthreads();
    if (n >= a.N) continue;
    const long long row = (long long)g * a.N + n;
    const float ws = a.fp8 ? a.w_scale[((long long)g * ((a.N + 127) / 128) + n / 128) * kb_count + kb]
                           : 1.f;
    for (int k = 0; k < kStep && kb * kStep + k < a.K; ++k) {
      const float w = value(a.weight, row * a.K + kb * kStep + k, a.fp8) * ws;
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc[i] = fmaf(xs[i][k], w, acc[i]);
    }
  }
  if (a.bias && n < a.N) {
    const float b = value(a.bias, (long long)g * a.N + n, false);
    for (int i = 0; i < kRows; ++i) acc[i] += b;
  }
}

__global__ void __launch_bounds__(kCols) linear_kernel(const LinearArgs a) {
  __shared__ float xs[kRows][kStep];
  __shared__ int found[3];
  if (threadIdx.x == 0) {
    int b = blockIdx.y, g = 0, lo = 0, hi = a.T;
    bool any = false;
    for (; g < a.G; ++g) {
      if (a.offsets) {
        lo = a.offsets[g];
        hi = a.offsets[g + 1];
        if (lo < 0 || hi < lo || hi > a.T) {
          record_status(a.status, GBMOE_ERR_DEVICE_CHECK);
          hi = lo;
        }
      }
      const int blocks = (hi - lo + kRows - 1) / kRows;
      if (b < blocks) {
        any = true;
        break;
      }
      b -= blocks;
    }
    found[0] = any ? g : -1;
    found[1] = lo + b * kRows;
    found[2] = min(kRows, hi - lo - b * kRows);
  }
  __syncthreads();
  const int g = found[0], r0 = found[1], rows = found[2];
  if (g < 0) return;
  const int c = blockIdx.x * kCols + threadIdx.x;
  float y[kRows];
  if (a.act == GBMOE_EPI_SILU_MUL) {
    float up[kRows];
    const int f = min(c, a.cols - 1);
    column(a, g, f, r0, rows, y, xs);
    column(a, g, a.cols + f, r0, rows, up, xs);
    for (int i = 0; i < kRows; ++i) y[i] = y[i] / (1.f + __expf(-y[i])) * up[i];
  } else {
    column(a, g, c, r0, rows, y, xs);
    for (int i = 0; i < kRows; ++i) y[i] = activated(y[i], a.act);
  }
  if (c >= a.cols) return;
  for (int i = 0; i < kRows; ++i) {
    if (i >= rows) break;
    const long long t = r0 + i;
    float v = y[i];
    if (a.row_weight) v *= a.row_weight[t];
    if (a.residual) v += value(a.residual, t * a.residual_stride + c, false);
    static_cast<__nv_bfloat16*>(a.out)[t * a.out_stride + c] = __float2bfloat16_rn(v);
  }
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
  const int blocks = (a.T + kRows - 1) / kRows + a.G - 1;
  linear_kernel<<<dim3((a.cols + kCols - 1) / kCols, blocks), kCols, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gbmoe
