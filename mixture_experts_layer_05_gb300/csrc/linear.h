// Launch interface of the dense and grouped products (moe_linear, moe_grouped_linear) between their
// C ABI (block_api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gbmoe.h"

namespace gbmoe {

constexpr int kLinearMaxGroups = 1024;

struct LinearArgs {
  const void* x;           // [T, K] bf16 or e4m3
  long long x_stride;
  const float* x_scale;    // e4m3: [K / 128, T]
  const void* weight;      // [G, N, K]
  const float* w_scale;    // e4m3: [G, ceil(N / 128), K / 128]
  const void* bias;        // [G, N] bf16, or NULL
  const void* residual;    // [T, cols] bf16, or NULL
  long long residual_stride;
  const float* row_weight;  // [T], or NULL
  void* out;               // [T, cols] bf16
  long long out_stride;
  const int* offsets;      // [G + 1] rows of each group, or NULL (one group of all rows)
  int T, G, K, N;
  int cols;                // output columns: N, or N / 2 with GBMOE_EPI_SILU_MUL
  int act;                 // gbmoe_epilogue_t
  bool fp8;
  int* status;             // or NULL
};
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream);

}  // namespace gbmoe
