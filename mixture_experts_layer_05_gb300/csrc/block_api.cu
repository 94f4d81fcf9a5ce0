// C ABI of the decoder-block operators around the layer: host-side checks, then one launch
// sequence each (norm.cu, kvappend.cu, attn.cu).
#include <climits>
#include <cmath>

#include "block.h"
#include "kernels.h"

#define GBMOE_API extern "C" __attribute__((visibility("default")))

namespace gbmoe {
namespace {

constexpr int kMaxRows = 1 << 22;
constexpr size_t kStatusBytes = 256;
// attention: the status region, then the counters of cut units
constexpr size_t kAttnHeadBytes = 1024;
static_assert(kStatusBytes + kAttnMaxCtas * sizeof(int) <= kAttnHeadBytes, "counters");

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

gbmoe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? GBMOE_OK : GBMOE_ERR_CUDA; }

gbmoe_status_t check_attn(const gbmoe_attn_config_t* c) {
  if (!c) return GBMOE_ERR_INVALID_ARG;
  if (c->num_q_heads < 1 || c->num_kv_heads < 1 || c->num_q_heads > 1024 ||
      c->num_q_heads % c->num_kv_heads || c->head_dim < 1 || c->page_size < 1 || c->window < 0 ||
      (c->cache_type != GBMOE_CACHE_BF16 && c->cache_type != GBMOE_CACHE_E4M3))
    return GBMOE_ERR_INVALID_ARG;
  // the append multiplies by 1 / scale
  auto scales = [](float x) { return std::isfinite(x) && x > 0.f && std::isfinite(1.f / x); };
  if (!std::isfinite(c->softmax_scale) || !(c->softmax_scale > 0.f) || !scales(c->k_scale) ||
      !scales(c->v_scale))
    return GBMOE_ERR_INVALID_ARG;
  if (c->cache_type == GBMOE_CACHE_BF16 && (c->k_scale != 1.f || c->v_scale != 1.f))
    return GBMOE_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->page_size < 8 || c->page_size > 1024 ||
      (c->page_size & (c->page_size - 1)))
    return GBMOE_ERR_UNSUPPORTED;
  return GBMOE_OK;
}

gbmoe_status_t check_paged(const gbmoe_attn_config_t& c, const gbmoe_paged_kv_t* kv) {
  if (!kv || !kv->k_cache || !kv->v_cache || !kv->block_table || !kv->cu_seqlens_q ||
      !kv->kv_lens || kv->num_pages < 1 || kv->num_seqs < 1 || kv->block_table_stride < 1 ||
      kv->page_stride < 1 || kv->token_stride < 1 || kv->head_stride < 1)
    return GBMOE_ERR_INVALID_ARG;
  if (kv->num_seqs > kAttnMaxSeqs) return GBMOE_ERR_UNSUPPORTED;
  const int64_t unit = c.cache_type == GBMOE_CACHE_E4M3 ? 16 : 8;  // elements per 16 bytes
  if (!aligned(kv->k_cache, 16) || !aligned(kv->v_cache, 16) || kv->page_stride % unit ||
      kv->token_stride % unit || kv->head_stride % unit || !aligned(kv->block_table, 4) ||
      !aligned(kv->cu_seqlens_q, 4) || !aligned(kv->kv_lens, 4))
    return GBMOE_ERR_INVALID_ARG;
  return GBMOE_OK;
}

PagedBatch batch_of(const gbmoe_attn_config_t& c, const gbmoe_paged_kv_t& kv, int T, int* status) {
  PagedBatch b;
  b.cu = kv.cu_seqlens_q;
  b.kv_lens = kv.kv_lens;
  b.table = kv.block_table;
  b.table_stride = kv.block_table_stride;
  b.S = kv.num_seqs;
  b.T = T;
  b.num_pages = kv.num_pages;
  b.page_shift = 0;
  while ((1 << b.page_shift) < c.page_size) ++b.page_shift;
  b.status = status;
  return b;
}

PagedCache cache_of(const gbmoe_paged_kv_t& kv) {
  return PagedCache{kv.k_cache, kv.v_cache, kv.page_stride, kv.token_stride, kv.head_stride};
}

}  // namespace
}  // namespace gbmoe

using namespace gbmoe;

GBMOE_API gbmoe_status_t moe_rms_norm(int32_t num_tokens, int32_t hidden_size,
                                      const gbmoe_rms_norm_args_t* args, gbmoe_stream_t stream) {
  if (num_tokens < 0 || num_tokens > kMaxRows || hidden_size < 1) return GBMOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return GBMOE_OK;
  if (!args || !args->x || !args->weight || (!args->y && !args->q) || (!args->q != !args->scale) ||
      (args->residual_out && !args->residual) || !std::isfinite(args->eps) || args->eps < 0.f)
    return GBMOE_ERR_INVALID_ARG;
  const int H = hidden_size;
  if (H % 8 || (args->q && H % kFp8Block) || H > rms_norm_max_hidden())
    return GBMOE_ERR_UNSUPPORTED;
  if (args->x_stride < H || args->x_stride % 8 ||
      (args->residual && (args->residual_stride < H || args->residual_stride % 8)) ||
      !aligned(args->x, 16) || !aligned(args->residual, 16) || !aligned(args->weight, 16) ||
      !aligned(args->y, 16) || !aligned(args->residual_out, 16) || !aligned(args->q, 16) ||
      !aligned(args->scale, 4))
    return GBMOE_ERR_INVALID_ARG;
  RmsNormArgs a;
  a.x = args->x;
  a.x_stride = args->x_stride;
  a.residual = args->residual;
  a.residual_stride = args->residual_stride;
  a.weight = args->weight;
  a.inv_h = 1.f / (float)H;
  a.eps = args->eps;
  a.y = args->y;
  a.residual_out = args->residual_out;
  a.q = args->q;
  a.scale = args->scale;
  a.T = num_tokens;
  a.H = H;
  PdlChain chain;
  return cuda_status(launch_rms_norm(a, (cudaStream_t)stream));
}

GBMOE_API gbmoe_status_t moe_kv_append(const gbmoe_attn_config_t* cfg, int32_t num_tokens,
                                       const gbmoe_paged_kv_t* kv,
                                       const gbmoe_kv_append_args_t* args,
                                       gbmoe_stream_t stream) {
  gbmoe_status_t s = check_attn(cfg);
  if (s != GBMOE_OK) return s;
  if (num_tokens < 0 || num_tokens > kMaxRows) return GBMOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return GBMOE_OK;
  s = check_paged(*cfg, kv);
  if (s != GBMOE_OK) return s;
  if (!args || !args->q || !args->k || !args->v || !args->q_out) return GBMOE_ERR_INVALID_ARG;
  const int64_t D = cfg->head_dim;
  if (args->q_stride < cfg->num_q_heads * D || args->q_stride % 8 ||
      args->k_stride < cfg->num_kv_heads * D || args->k_stride % 8 ||
      args->v_stride < cfg->num_kv_heads * D || args->v_stride % 8 || !aligned(args->q, 16) ||
      !aligned(args->k, 16) || !aligned(args->v, 16) || !aligned(args->q_out, 16) ||
      !aligned(args->cos_sin, 16) || !aligned(args->workspace, kStatusBytes))
    return GBMOE_ERR_INVALID_ARG;
  if (args->rotary_dim < 0 || args->rotary_dim > D || args->rotary_dim % 16 ||
      (args->rotary_dim > 0) != (args->cos_sin != nullptr) ||
      (args->cos_sin && args->max_position < 1))
    return GBMOE_ERR_INVALID_ARG;
  KvAppendArgs a;
  a.b = batch_of(*cfg, *kv, num_tokens, static_cast<int*>(args->workspace));
  a.c = cache_of(*kv);
  a.q = args->q;
  a.k = args->k;
  a.v = args->v;
  a.q_stride = args->q_stride;
  a.k_stride = args->k_stride;
  a.v_stride = args->v_stride;
  a.cos_sin = args->cos_sin;
  a.max_pos = args->max_position;
  a.rotary = args->rotary_dim;
  a.interleaved = args->interleaved != 0;
  a.q_out = args->q_out;
  a.hq = cfg->num_q_heads;
  a.hkv = cfg->num_kv_heads;
  a.D = cfg->head_dim;
  a.fp8 = cfg->cache_type == GBMOE_CACHE_E4M3;
  a.k_scale = cfg->k_scale;
  a.v_scale = cfg->v_scale;
  a.k_inv = 1.f / cfg->k_scale;
  a.v_inv = 1.f / cfg->v_scale;
  PdlChain chain;
  return cuda_status(launch_kv_append(a, (cudaStream_t)stream));
}

GBMOE_API size_t moe_paged_attention_workspace_size(const gbmoe_attn_config_t* cfg) {
  if (check_attn(cfg) != GBMOE_OK) return 0;
  return kAttnHeadBytes + attn_scratch_bytes(cfg->head_dim);
}

GBMOE_API gbmoe_status_t moe_paged_attention(const gbmoe_attn_config_t* cfg, int32_t num_tokens,
                                             const gbmoe_paged_kv_t* kv, const void* q,
                                             int64_t q_stride, void* out, float* lse,
                                             void* workspace, size_t workspace_bytes,
                                             gbmoe_stream_t stream) {
  gbmoe_status_t s = check_attn(cfg);
  if (s != GBMOE_OK) return s;
  if (num_tokens < 0 || num_tokens > kMaxRows) return GBMOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return GBMOE_OK;
  if ((int64_t)num_tokens * cfg->num_q_heads > (1 << 30)) return GBMOE_ERR_UNSUPPORTED;
  s = check_paged(*cfg, kv);
  if (s != GBMOE_OK) return s;
  if (!q || !out || q_stride < (int64_t)cfg->num_q_heads * cfg->head_dim || q_stride % 8 ||
      !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return GBMOE_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kStatusBytes) ||
      workspace_bytes < moe_paged_attention_workspace_size(cfg))
    return GBMOE_ERR_WORKSPACE;
  AttnArgs a;
  a.b = batch_of(*cfg, *kv, num_tokens, static_cast<int*>(workspace));
  a.c = cache_of(*kv);
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.hq = cfg->num_q_heads;
  a.hkv = cfg->num_kv_heads;
  a.D = cfg->head_dim;
  a.fp8 = cfg->cache_type == GBMOE_CACHE_E4M3;
  a.causal = cfg->causal != 0;
  a.window = cfg->window;
  a.scale_log2 = cfg->softmax_scale * cfg->k_scale * 1.4426950408889634f;
  a.v_scale = cfg->v_scale;
  a.counters = reinterpret_cast<int*>(static_cast<char*>(workspace) + kStatusBytes);
  a.scratch = static_cast<char*>(workspace) + kAttnHeadBytes;
  if (!attn_fits(a)) return GBMOE_ERR_UNSUPPORTED;
  PdlChain chain;
  return cuda_status(launch_attn(a, (cudaStream_t)stream));
}
