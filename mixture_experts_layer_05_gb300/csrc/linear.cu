// The choice between the kernels of moe_linear and moe_grouped_linear, and how a call is cut.
#include "linear.cuh"

namespace gbmoe {

namespace {

bool encode(const LinearArgs& a, CUtensorMap* m, const void* p, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  auto enc = tensor_map_encoder();
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc && enc(m, a.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                    const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows of `cols` elements, `stride` apart, in boxes of 128 bytes by box_rows
bool map_rows(const LinearArgs& a, CUtensorMap* m, const void* p, cuuint64_t rows, cuuint64_t stride,
              int box_rows) {
  const cuuint64_t es = a.fp8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)a.K, rows}, strides[1] = {stride * es};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows};
  return encode(a, m, p, 2, dims, strides, box);
}

}  // namespace

bool lin_map_rows(const LinearArgs& a, CUtensorMap* w, CUtensorMap* x, int x_box) {
  return map_rows(a, w, a.weight, (cuuint64_t)a.G * a.N, a.K, kLinWRows) &&
         map_rows(a, x, a.x, a.T, a.x_stride, x_box);
}

bool lin_maps(const LinearArgs& a, int x_box, CUtensorMap* w, CUtensorMap* x) {
  if (a.act != GBMOE_EPI_SILU_MUL) return lin_map_rows(a, w, x, x_box);
  // (k, row of 16, gate or up, block of 16 features, group): 16 gate rows, their 16 up rows, ...
  const cuuint64_t es = a.fp8 ? 1 : 2, K = a.K, N = a.N, I = N / 2;
  const cuuint64_t dims[5] = {K, 16, 2, I / 16, (cuuint64_t)a.G};
  const cuuint64_t strides[4] = {K * es, I * K * es, 16 * K * es, N * K * es};
  const cuuint32_t box[5] = {(cuuint32_t)(128 / es), 16, 2, 4, 1};
  return encode(a, w, a.weight, 5, dims, strides, box) && map_rows(a, x, a.x, a.T, a.x_stride, x_box);
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
  if (pair && a.fp8) {
    L.bn = 128;
    L.n_tiles = ceil_div(a.cols, 2 * cols);
    L.gm = 16;
    const long long units = ((long long)ceil_div(a.T, L.bn) + groups - 1) * L.n_tiles;
    return launch_linear_fp8(L, units > 4096 ? 4096 : (int)units, stream);
  }
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
