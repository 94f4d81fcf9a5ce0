// Launch interface of the decoder-block operators around the MoE layer (norm, cache append,
// paged attention) between their C ABI (block_api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gbmoe.h"

namespace gbmoe {

// The sequences of one call: packed new tokens (cu), total lengths, and their pages.
struct PagedBatch {
  const int* cu;         // [S + 1] first new token of each sequence
  const int* kv_lens;    // [S] keys of each sequence, its new tokens among them
  const int* table;      // [S, table_stride] page ids
  int table_stride;
  int S, T;
  int num_pages;
  int page_shift;        // page_size = 1 << page_shift
  int* status;
};

// A paged K or V: element (page, row, head, d) at page * page_stride + row * token_stride +
// head * head_stride + d.
struct PagedCache {
  void* k;
  void* v;
  long long page_stride, token_stride, head_stride;
};

struct RmsNormArgs {
  const void* x;
  long long x_stride;
  const void* residual;
  long long residual_stride;
  const void* weight;
  float eps, inv_h;      // inv_h = 1 / H
  void* y;
  void* residual_out;
  uint8_t* q;
  float* scale;
  int T, H;
};
cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t stream);
int rms_norm_max_hidden();

// The FP8 layer's gather of rows that are quantized already: codes q [T, H] and scales
// s [H / 128, T] of token f / k to row inv[f] of x_perm_q and xs_perm (group stride perm_ld).
cudaError_t launch_gather_fp8(const uint8_t* q, const float* s, int H, const int* inv, int n,
                              int k, int T, uint8_t* x_perm_q, float* xs_perm, int perm_ld,
                              cudaStream_t stream);

struct KvAppendArgs {
  PagedBatch b;
  PagedCache c;
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const float* cos_sin;                    // [max_pos, rotary] (R / 2 cosines, R / 2 sines)
  int max_pos, rotary, interleaved;
  void* q_out;
  int hq, hkv, D;
  bool fp8;
  float k_scale, v_scale;
  float k_inv, v_inv;    // 1 / scale
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream);

struct AttnArgs {
  PagedBatch b;
  PagedCache c;
  const void* q;
  long long q_stride;
  void* out;
  float* lse;            // or NULL
  int hq, hkv, D;
  bool fp8, causal;
  int window;
  float scale_log2;      // softmax scale * k_scale * log2(e)
  float v_scale;
  int* counters;         // kAttnMaxCtas, zero between calls
  void* scratch;
};
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream);
bool attn_fits(const AttnArgs& a);  // whether the call's work can be counted
size_t attn_scratch_bytes(int D);
constexpr int kAttnMaxSeqs = 8192;
constexpr int kAttnMaxCtas = 160;  // workspace bound; the kernels run one CTA per SM

}  // namespace gbmoe
