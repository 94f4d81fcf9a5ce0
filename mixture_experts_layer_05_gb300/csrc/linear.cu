// The choice between the kernels of moe_linear and moe_grouped_linear, and how a call is cut.
#include "linear.cuh"

namespace gbmoe {

bool lin_maps(const LinearArgs& a, int x_box, CUtensorMap* w, CUtensorMap* x) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const CUtensorMapDataType type =
      a.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t es = a.fp8 ? 1 : 2, K = a.K, N = a.N, G = a.G;
  const cuuint32_t inner = (cuuint32_t)(128 / es), one[5] = {1, 1, 1, 1, 1};
  auto make = [&](CUtensorMap* m, const void* p, int rank, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box) {
    return enc(m, type, rank, const_cast<void*>(p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (a.act == GBMOE_EPI_SILU_MUL) {
    // (k, row of 16, gate or up, block of 16 features, group): 16 gate rows, their 16 up rows, ...
    const cuuint64_t I = N / 2;
    const cuuint64_t dims[5] = {K, 16, 2, I / 16, G};
    const cuuint64_t strides[4] = {K * es, I * K * es, 16 * K * es, N * K * es};
    const cuuint32_t box[5] = {inner, 16, 2, 4, 1};
    if (!make(w, a.weight, 5, dims, strides, box)) return false;
  } else {
    const cuuint64_t dims[2] = {K, G * N}, strides[1] = {K * es};
    const cuuint32_t box[2] = {inner, kLinWRows};
    if (!make(w, a.weight, 2, dims, strides, box)) return false;
  }
  const cuuint64_t dims[2] = {K, (cuuint64_t)a.T}, strides[1] = {(cuuint64_t)a.x_stride * es};
  const cuuint32_t box[2] = {inner, (cuuint32_t)x_box};
  return make(x, a.x, 2, dims, strides, box);
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
  LinLaunch L = {};
  L.a = a;
  L.k_blocks = (a.K * (a.fp8 ? 1 : 2) + 127) / 128;
  const int cols = a.act == GBMOE_EPI_SILU_MUL ? 64 : 128;   // output columns of 128 weight rows
  auto ceil_div = [](long long x, long long y) { return (int)((x + y - 1) / y); };
  const int mean = ceil_div(a.T, a.G);
  const int groups = a.G < a.T ? a.G : a.T;                  // with rows, at most
  const bool pair = mean > 128;
  if (pair) {
    int bn = ceil_div(mean, ceil_div(mean, 256));
    bn = (bn + 31) & ~31;
      L.bn = bn;
    L.n_tiles = ceil_div(a.cols, 2 * cols);
    L.gm = 16;
    const long long units = ((long long)ceil_div(a.T, L.bn) + groups - 1) * L.n_tiles;
    return launch_linear_pair(L, units > 4096 ? 4096 : (int)units, stream);
  }
  int bn = ceil_div(mean, ceil_div(mean, 128));
  bn = (bn + 15) & ~15;
  L.bn = bn;
  L.n_tiles = ceil_div(a.cols, cols);
  L.gm = 1 << 16;
  const long long units = ((long long)ceil_div(a.T, L.bn) + groups - 1) * L.n_tiles;
  // the cluster: as many CTAs a unit as the units leave free
  int best = 1;
  double best_cost = 1e30;
  for (int C = 1; C <= 8 && C <= L.k_blocks; ++C) {
    const int room = num_sms() / C;
    const double cost = ceil_div(units, room) * (ceil_div(L.k_blocks, C) + (C > 1 ? 4 : 2));
    if (cost < best_cost * 0.999) {
      best_cost = cost;
      best = C;
    }
  }
  return launch_linear_stream(L, best, units > 4096 ? 4096 : (int)units, stream);
}

}  // namespace gbmoe
