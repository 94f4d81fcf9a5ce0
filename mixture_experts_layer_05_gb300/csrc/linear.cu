// Tensor maps of moe_linear and moe_grouped_linear, and the launch that linear_plan.h chose for a call.
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

// `rows` rows of K elements, `stride` elements apart.
bool map_rows(const LinearArgs& a, CUtensorMap* m, const void* p, cuuint64_t rows, cuuint64_t stride,
              int box_rows, int kps) {
  const cuuint64_t es = a.fp8 ? 1 : 2, inner = 128 / es, K = a.K;
  const bool whole = kps > 0;
  const cuuint64_t dims[3] = {whole ? inner : K, rows, whole ? K / inner : 1};
  const cuuint64_t strides[2] = {stride * es, 128};
  const cuuint32_t box[3] = {(cuuint32_t)inner, (cuuint32_t)box_rows, (cuuint32_t)(whole ? kps : 1)};
  return encode(a, m, p, 3, dims, strides, box);
}

}  // namespace

bool lin_map_x(const LinearArgs& a, int rows, int kps, CUtensorMap* x) {
  return map_rows(a, x, a.x, a.T, a.x_stride, rows, kps);
}

bool lin_map_rows(const LinearArgs& a, int rows, int kps, CUtensorMap* w) {
  return map_rows(a, w, a.weight, (cuuint64_t)a.G * a.N, a.K, rows, kps);
}

bool lin_map_tiles(const LinearArgs& a, int rows, int kps, CUtensorMap* w) {
  if (a.act != GBMOE_EPI_SILU_MUL) return lin_map_rows(a, rows, kps, w);
  // (k, row of 16, gate or up of each group, block of 16 features, K block)
  const cuuint64_t es = a.fp8 ? 1 : 2, inner = 128 / es, K = a.K, I = a.N / 2;
  const bool whole = kps > 0;
  const cuuint64_t dims[5] = {whole ? inner : K, 16, 2 * (cuuint64_t)a.G, I / 16, whole ? K / inner : 1};
  const cuuint64_t strides[4] = {K * es, I * K * es, 16 * K * es, 128};
  const cuuint32_t box[5] = {(cuuint32_t)inner, 16, 2, (cuuint32_t)rows / 32, (cuuint32_t)(whole ? kps : 1)};
  return encode(a, w, a.weight, 5, dims, strides, box);
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
  LinLaunch L = {};
  L.a = a;
  L.k_blocks = (a.K * (a.fp8 ? 1 : 2) + 127) / 128;
  const LinSize size = {a.T, a.G, a.K, a.N, a.offsets != nullptr, a.act == GBMOE_EPI_SILU_MUL, a.fp8};
  const LinPlan p = lin_plan(size, num_sms(), [&](int bn, int C) { return linear_stream_room(a, bn, C); });
  if (!p.ok) return cudaErrorInvalidConfiguration;
  L.bn = p.bn;
  L.n_tiles = p.n_tiles;
  if (p.many) {
    L.gm = 16;
    return a.fp8 ? launch_linear_fp8(L, p.units, stream) : launch_linear_pair(L, p.units, stream);
  }
  L.gm = 1 << 16;
  L.cluster = p.cluster;
  L.choices = p.choices;
  for (int i = 0; i < p.choices; ++i) L.rows[i] = p.rows[i];
  return launch_linear_stream(L, p.units, stream);
}

}  // namespace gbmoe
