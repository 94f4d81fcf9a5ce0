/*
 * gbmoe.h: C ABI of the GB300 (sm_103a) FusedMoE layer forward.
 *
 * The forward is the one the vLLM `fused_moe/layer` page builds around
 * `FusedMoE` (constructor arguments, `select_experts`, `forward_impl`) and the
 * sglang `fused_moe_triton/layer.py` page runs in one call
 * (`FlashInferFusedMoE.forward_impl`: router logits, correction bias, hidden
 * states and both expert weight stacks in, the combined output out), with the
 * DeepSeek shared expert of the sglang `models/deepseek_v2.py` page
 * (`DeepseekV2MoE.forward_normal`) added on top.
 *
 * Conventions for every entry point
 *  - All array pointers are DEVICE pointers owned by the caller. The library
 *    never allocates, frees or keeps them; scratch lives in a caller-provided
 *    workspace whose size the matching *_workspace_size() call returns.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default
 *    stream) and the call returns without synchronising. Outputs are valid once
 *    the stream reaches that point.
 *  - Arguments are validated on the host before anything is enqueued; a
 *    negative status means nothing was enqueued (except GBMOE_ERR_CUDA, which
 *    reports a failed launch). Kernels never trap: a failed device-side check or a
 *    bounded wait that ran out is recorded in the int32 status word at the start
 *    of the workspace, read (and reset) with moe_get_device_status(). The word
 *    keeps the first error since its last reset, so a new workspace must start
 *    with its first 256 bytes zeroed.
 *  - bf16 tensors are passed as `const void*` (IEEE bfloat16, row-major).
 *  - num_tokens == 0 is a successful no-op (the empty-batch early return of
 *    `DeepseekV2MoE.forward_normal`).
 */
#ifndef GBMOE_H
#define GBMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* gbmoe_stream_t; /* identical to cudaStream_t */

typedef enum {
  GBMOE_OK = 0,
  GBMOE_ERR_INVALID_ARG = -1,   /* null pointer, bad size, inconsistent flags */
  GBMOE_ERR_UNSUPPORTED = -2,   /* valid for the method, not built here (see each call) */
  GBMOE_ERR_WORKSPACE = -3,     /* workspace null or smaller than *_workspace_size() */
  GBMOE_ERR_CUDA = -4,          /* a CUDA runtime call or launch failed */
  GBMOE_ERR_DEVICE_CHECK = -5,  /* a device-side bounds check failed */
  GBMOE_ERR_TIMEOUT = -6        /* a device-side bounded wait ran out */
} gbmoe_status_t;

typedef enum { GBMOE_SCORE_SOFTMAX = 0, GBMOE_SCORE_SIGMOID = 1 } gbmoe_scoring_t;
typedef enum { GBMOE_ACT_SILU = 0 } gbmoe_act_t;
typedef enum {
  GBMOE_QUANT_NONE = 0,
  GBMOE_QUANT_FP8_BLOCK128 = 1,
  GBMOE_QUANT_NVFP4 = 2
} gbmoe_weight_quant_t;

/*
 * Layer configuration; field names follow the FusedMoE constructor (vLLM
 * `fused_moe/layer` page, `FusedMoE.__init__`) and `DeepseekV2MoE.__init__`
 * (sglang `models/deepseek_v2.py` page) for the shared expert.
 *
 *  num_experts            E, routed experts (1..1024)
 *  top_k                  k, experts per token (1..min(E, 32))
 *  hidden_size            H, a multiple of 128
 *  intermediate_size      I, a multiple of 128
 *  renormalize            !=0: divide the chosen weights by their sum
 *  use_grouped_topk       !=0: group-limited routing (num_expert_group,
 *                         topk_group required; E % num_expert_group == 0,
 *                         num_expert_group <= 32, topk_group <= num_expert_group,
 *                         top_k <= topk_group * E / num_expert_group)
 *  scoring_func           gbmoe_scoring_t; SIGMOID requires use_grouped_topk
 *                         (the constructor rejects non-softmax ungrouped routing)
 *  routed_scaling_factor  multiplies every routed weight (not the shared expert)
 *  activation             must be GBMOE_ACT_SILU (else UNSUPPORTED)
 *  is_act_and_mul         1: gated, w13 [E, 2I, H], act = silu-gate * up;
 *                         0: not gated (`is_gated=False`), w13 [E, I, H], act = silu(z)
 *  shared_intermediate_size  I_s of the dense shared SwiGLU expert; 0 = none;
 *                         else a multiple of 128 (gated routed experts only)
 *  swiglu_limit           > 0: clamp the gate to <= L and the up half to [-L, L]
 *                         before the activation (`swiglu_limit`, `gemm1_clamp_limit`;
 *                         also applied to the shared expert); 0 = no clamp
 *  gemm1_alpha            gated act = g * sigmoid(alpha * g) * u for the routed experts
 *                         (`gemm1_alpha`); 0 means 1
 *  apply_router_weight_on_input  != 0: the routing weight scales the expert's input
 *                         rows instead of its output (FusedMoE constructor argument)
 * The pages name the last three options without their arithmetic; the reading used is
 * the one the NPU clipped-SwiGLU call's arguments (alpha, limit, bias) point to.
 *  weight_quant           gbmoe_weight_quant_t. FP8_BLOCK128: the w8a8 fp8 layer of the
 *                         sglang `models/deepseek_v2.py` page (`DeepseekV2MoE`'s
 *                         quant-once path, `DeepseekV2MLP.forward`'s fp8 down GEMM):
 *                         expert and shared weights are e4m3fn bytes with one fp32 scale
 *                         per 128 x 128 block (w = q * scale[n / 128][k / 128]); the input
 *                         is quantized once per token and group of 128 hidden columns
 *                         (s = max(amax, 1e-10) / 448, q = e4m3(x / s), fp32), feeds the
 *                         routed and the shared experts, and each act is quantized the
 *                         same way before its w2 GEMM. Requires H % 256 == 0, gated SiLU
 *                         without clamp or alpha, no expert biases, no
 *                         apply_router_weight_on_input (else UNSUPPORTED).
 *                         NVFP4: the w4a4 layer of FlashInferFP4MoE (sglang
 *                         `fused_moe_triton/layer.py` page, `trtllm_fp4_block_scale_moe`):
 *                         weights are e2m1 codes with one e4m3 scale per 16 values along K
 *                         and a per-expert fp32 weight_scale_2 (w = q * sf * s2), passed in
 *                         the layout moe_nvfp4_prepare_weight writes; the input is quantized
 *                         per token and block of 16 with the per-tensor input_scale g
 *                         (sf = e4m3(g * amax / 6), q = e2m1(x * g / sf), fp32 steps;
 *                         dequantized q * sf / g), and each act the same way with act_scale
 *                         before its w2 GEMM (moe_quant_nvfp4 is that quantization alone).
 *                         Same restrictions as FP8_BLOCK128 (H % 128 suffices). The pages'
 *                         layer casts e_score_correction_bias to the activations' dtype
 *                         before routing; callers wanting that pass bf16-valued biases.
 */
typedef struct {
  int32_t num_experts;
  int32_t top_k;
  int32_t hidden_size;
  int32_t intermediate_size;
  int32_t renormalize;
  int32_t use_grouped_topk;
  int32_t num_expert_group;
  int32_t topk_group;
  int32_t scoring_func;
  float routed_scaling_factor;
  int32_t activation;
  int32_t is_act_and_mul;
  int32_t shared_intermediate_size;
  float swiglu_limit;
  float gemm1_alpha;
  int32_t apply_router_weight_on_input;
  int32_t weight_quant;
} gbmoe_config_t;

/*
 * moe_topk: router scoring and (grouped) top-k.
 * Defined by `FusedMoE.select_experts` (vLLM `fused_moe/layer` page): the
 * grouped_topk branch (num_expert_group, topk_group, scoring_func,
 * routed_scaling_factor, e_score_correction_bias), the biased fused_topk_bias
 * branch and the plain fused_topk branch.
 *  - score s = softmax(logits row) or sigmoid(logits); key q = s + bias when
 *    `e_score_correction_bias` is non-NULL, else q = s.
 *  - grouped: the topk_group groups (contiguous runs of E/num_expert_group
 *    experts) with the largest group score survive; the group score is the
 *    largest s in the group without a bias and the sum of the two largest q in
 *    the group with one.
 *  - the top_k largest q among surviving experts (ties to the lower index), in
 *    descending q order; weight = s of that expert, divided by the sum of the
 *    chosen s if renormalize, then times routed_scaling_factor.
 * router_logits [T, E] fp32; e_score_correction_bias [E] fp32 or NULL;
 * topk_weights [T, top_k] fp32 (out); topk_ids [T, top_k] int32 (out).
 * Errors: INVALID_ARG (nulls, sizes, group arguments), UNSUPPORTED (sigmoid
 * without grouping).
 */
gbmoe_status_t moe_topk(const gbmoe_config_t* cfg, int32_t num_tokens,
                        const float* router_logits, const float* e_score_correction_bias,
                        float* topk_weights, int32_t* topk_ids, gbmoe_stream_t stream);

/*
 * moe_align_block_size: group the (token, slot) pairs by expert, padded to
 * block_size, for the grouped expert GEMMs of the FusedMoE forward (the
 * Triton fused_moe path behind `UnquantizedFusedMoEMethod` on the vLLM
 * `fused_moe/layer` page).
 *  - flat index f = t*top_k + j of topk_ids [T, top_k] (int32, values in [0, E));
 *  - experts in ascending order, each expert's flat indices ascending (stable),
 *    each run padded with the sentinel T*top_k to a multiple of block_size;
 *  - sorted_token_ids [T*top_k + E*(block_size-1)] int32 (out; entries past
 *    num_tokens_post_padded are unspecified);
 *  - expert_ids [(T*top_k + E*(block_size-1)) / block_size + 1] int32 (out;
 *    one per block; entries past num_tokens_post_padded/block_size are -1);
 *  - num_tokens_post_padded [1] int32 (out) = sum over experts of the padded runs.
 * block_size: 1..1024. Workspace: moe_align_block_size_workspace_size().
 * A topk_id outside [0, E) sets GBMOE_ERR_DEVICE_CHECK in the device status and
 * is counted as expert 0.
 */
size_t moe_align_block_size_workspace_size(int32_t num_tokens, int32_t top_k, int32_t num_experts);
gbmoe_status_t moe_align_block_size(const int32_t* topk_ids, int32_t num_tokens, int32_t top_k,
                                    int32_t num_experts, int32_t block_size,
                                    int32_t* sorted_token_ids, int32_t* expert_ids,
                                    int32_t* num_tokens_post_padded, void* workspace,
                                    size_t workspace_bytes, gbmoe_stream_t stream);

/*
 * moe_align_block_size_no_workspace: moe_align_block_size for callers that cannot
 * allocate device memory. The pages have no counterpart; this entry point exists for
 * the deployment, not the method. Plugins hosted by a framework that owns and
 * pre-plans every device allocation (an inference server with a fixed memory pool, a
 * runtime whose extensions may not call cudaMalloc) have no workspace to pass, so
 * this variant keeps its scratch in a fixed 1 MiB device array inside the library and
 * allocates nothing. Same arguments and outputs as moe_align_block_size, minus the
 * workspace.
 *  - Limit: requests needing more than 1 MiB of scratch
 *    (2 * ceil(T*top_k / 2048) * num_experts * 4 bytes) return GBMOE_ERR_WORKSPACE.
 *  - The array is shared by every call on a device and keeps the last call's
 *    contents; each call overwrites what it reads, so nothing must start at zero.
 *    Calls that overlap on the GPU (unordered streams) race on it: do not issue them.
 *  - The first call on a device looks up the array's device address with that device
 *    current; make that first call before any stream capture.
 *  - No status word: a topk_id outside [0, E) is counted as expert 0, unreported.
 */
gbmoe_status_t moe_align_block_size_no_workspace(const int32_t* topk_ids, int32_t num_tokens,
                                                 int32_t top_k, int32_t num_experts,
                                                 int32_t block_size, int32_t* sorted_token_ids,
                                                 int32_t* expert_ids,
                                                 int32_t* num_tokens_post_padded,
                                                 gbmoe_stream_t stream);

/*
 * moe_forward: the whole layer, from router logits to the combined output.
 *  1. moe_topk (above);
 *  2. align by expert (above) with the block size moe_forward_block_size(),
 *     and gather the hidden rows into expert order;
 *  3. per block: [gate | up] = x_rows @ w13[e]^T, act = silu(gate) * up
 *     (`SiluAndMul` of `DeepseekV2MLP`; w13 rows [0, I) gate, [I, 2I) up as
 *     `FusedMoE._load_w13` lays them out), rounded to bf16;
 *  4. o = act @ w2[e]^T, times the token's routing weight;
 *  5. y[t] = sum over j ascending of the weighted o[t, j], plus the shared expert
 *     silu(x W1s^T) * (x W3s^T) W2s^T unscaled (`DeepseekV2MoE.forward_normal`),
 *     accumulated in fp32 and rounded once to bf16.
 * hidden_states [T, H] bf16; router_logits [T, E] fp32; bias [E] fp32 or NULL;
 * w13_weight [E, 2I, H] bf16; w2_weight [E, H, I] bf16; shared_w13 [2I_s, H] and
 * shared_w2 [H, I_s] bf16 (both NULL iff cfg->shared_intermediate_size == 0);
 * output [T, H] bf16 (out). All bf16 pointers 16-byte aligned.
 * Workspace: moe_forward_workspace_size(cfg, max_tokens) bytes, 256-byte
 * aligned, for any num_tokens <= max_tokens; its layout is reported by
 * moe_forward_workspace_layout().
 */
size_t moe_forward_workspace_size(const gbmoe_config_t* cfg, int32_t max_num_tokens);
int32_t moe_forward_block_size(const gbmoe_config_t* cfg, int32_t num_tokens);
gbmoe_status_t moe_forward(const gbmoe_config_t* cfg, int32_t num_tokens,
                           const void* hidden_states, const float* router_logits,
                           const float* e_score_correction_bias, const void* w13_weight,
                           const void* w2_weight, const void* shared_w13, const void* shared_w2,
                           void* output, void* workspace, size_t workspace_bytes,
                           gbmoe_stream_t stream);

/*
 * moe_forward_events: moe_forward that also records caller-created CUDA events
 * (cudaEvent_t, passed as void*) on `stream` at the stage boundaries:
 * events[0] before routing, [1] after routing + align + gather, [2] after the
 * w13 GEMMs, [3] after the w2 GEMMs, [4] after the combine; a NULL entry is
 * skipped. The records are external (cudaEventRecordExternal): inside a stream
 * capture they become event-record nodes that time each replay. `events` may be
 * NULL (then identical to moe_forward); num_events must then be 0, else 5.
 */
#define GBMOE_NUM_STAGE_EVENTS 5
gbmoe_status_t moe_forward_events(const gbmoe_config_t* cfg, int32_t num_tokens,
                                  const void* hidden_states, const float* router_logits,
                                  const float* e_score_correction_bias, const void* w13_weight,
                                  const void* w2_weight, const void* shared_w13,
                                  const void* shared_w2, void* output, void* workspace,
                                  size_t workspace_bytes, void* const* events, int32_t num_events,
                                  gbmoe_stream_t stream);

/*
 * moe_forward_ex: moe_forward with every tensor in one struct, plus the per-expert
 * biases of the FusedMoE `with_bias` / `has_bias` option (sglang
 * `fused_moe_triton/layer.py` page: `w13_weight_bias`, `w2_weight_bias`):
 *   [gate | up] = x @ w13[e]^T + w13_bias[e]   (w13_bias [E, 2I] bf16; [E, I] not gated)
 *   o = act @ w2[e]^T + w2_bias[e]              (w2_bias [E, H] bf16)
 * Either bias may be NULL; the shared expert has none. events / num_events as in
 * moe_forward_events (NULL / 0 for none).
 */
typedef struct {
  const void* hidden_states;
  const float* router_logits;
  const float* e_score_correction_bias;
  const void* w13_weight;
  const void* w2_weight;
  const void* shared_w13;
  const void* shared_w2;
  const void* w13_bias;
  const void* w2_bias;
  void* output;
  void* workspace;
  size_t workspace_bytes;
  void* const* events;
  int32_t num_events;
  const void* gate_weight;   /* [E, H] bf16: when router_logits is NULL, the logits are
                                computed first as hidden_states @ gate_weight^T with fp32
                                sums (`MoEGate.forward`); exactly one of the two is given.
                                Batches of at most 16 tokens compute them inside the routing
                                launch (no [T, E] logits pass of their own), larger ones with
                                the tensor-core GEMM of moe_router_logits. Uses the int32 at
                                byte 4 of the workspace as an arrival counter (zero between
                                calls, like the status word) */
  /* weight_quant == FP8_BLOCK128 only (else NULL): the weights above are e4m3fn bytes and
     these their fp32 block scales, row-major per matrix:
     w13_scale [E, 2I/128, H/128], w2_scale [E, H/128, I/128],
     shared_w13_scale [2I_s/128, H/128], shared_w2_scale [H/128, I_s/128] */
  const float* w13_scale;
  const float* w2_scale;
  const float* shared_w13_scale;
  const float* shared_w2_scale;
  /* weight_quant == NVFP4 only (else NULL / 0): w13_weight, w2_weight, shared_w13 and
     shared_w2 are prepared NVFP4 weights (moe_nvfp4_prepare_weight of the [E * 2I, H],
     [E * H, I], [2 I_s, H] and [H, I_s] stacks); these their fp32 per-expert scales
     (device): w13_weight_scale_2 [E], w2_weight_scale_2 [E], shared_weight_scale_2 [2]
     (w13, w2); and the per-tensor scales (host values > 0) of the input's and the act's
     quantization, routed and shared */
  const float* w13_weight_scale_2;
  const float* w2_weight_scale_2;
  const float* shared_weight_scale_2;
  float input_scale;
  float act_scale;
  float shared_input_scale;
  float shared_act_scale;
} gbmoe_forward_args_t;
gbmoe_status_t moe_forward_ex(const gbmoe_config_t* cfg, int32_t num_tokens,
                              const gbmoe_forward_args_t* args, gbmoe_stream_t stream);

/*
 * moe_forward_q: moe_forward_ex of the FP8_BLOCK128 layer whose input is quantized already, as
 * moe_rms_norm writes it: hidden_q [T, H] e4m3fn bytes (16-byte aligned) and hidden_scale
 * [H / 128, T] fp32 take the place of the layer's own quantization of hidden_states, which only
 * the router GEMM still reads (args->hidden_states may be NULL when router_logits is given).
 * With the outputs of moe_quant_fp8_per_token_group the result is moe_forward_ex's, bit for bit.
 * UNSUPPORTED for other layers.
 */
gbmoe_status_t moe_forward_q(const gbmoe_config_t* cfg, int32_t num_tokens,
                             const gbmoe_forward_args_t* args, const uint8_t* hidden_q,
                             const float* hidden_scale, gbmoe_stream_t stream);

/*
 * moe_router_logits: the router GEMM in front of the layer, `MoEGate.forward` on the
 * sglang `models/deepseek_v2.py` page: router_logits [T, E] fp32 = hidden_states
 * [T, H] bf16 @ gate_weight [E, H]^T bf16, fp32 accumulation on the tensor cores.
 * H a multiple of 64, 1 <= E <= 1024, pointers 16-byte aligned, T = 0 a no-op.
 */
gbmoe_status_t moe_router_logits(int32_t num_tokens, int32_t hidden_size, int32_t num_experts,
                                 const void* hidden_states, const void* gate_weight,
                                 float* router_logits, gbmoe_stream_t stream);

/*
 * moe_quant_fp8_per_token_group: the per-token-group-128 fp8 quant of bf16 rows that the
 * FP8_BLOCK128 layer applies to its input (sglang `models/deepseek_v2.py` page,
 * `DeepseekV2MoE._maybe_quant_moe_input_once`): for each row r and group g of 128
 * consecutive columns, s = max(max |x|, 1e-10) / 448 and q = e4m3fn(x / s), both one fp32
 * division, the conversion round-to-nearest-even saturating at +-448.
 *   x      [num_rows, hidden_size] bf16, device, 16-byte aligned
 *   q      [num_rows, hidden_size] e4m3fn bytes, device (written)
 *   scale  [hidden_size / 128, num_rows] fp32, device, group-major ("column-major
 *          scales"): scale[g * num_rows + r] (written)
 * hidden_size a positive multiple of 128; num_rows = 0 is a no-op. Asynchronous on
 * `stream`; INVALID_ARG for bad sizes or pointers.
 */
gbmoe_status_t moe_quant_fp8_per_token_group(int32_t num_rows, int32_t hidden_size,
                                             const void* x, uint8_t* q, float* scale,
                                             gbmoe_stream_t stream);

/*
 * moe_quant_nvfp4: fp4_quantize(x, global_scale, 16) as the FlashInferFP4MoE layer applies
 * it to its input (sglang `fused_moe_triton/layer.py` page, `_quantize_hidden_states_fp4`):
 * for each row and block of 16 consecutive columns, amax = max |x|, sf = e4m3(g * (amax /
 * 6)) (round to nearest even, saturating at 448), r = g / sf (0 when sf is 0), q =
 * e2m1(x * r) (round to nearest even, saturating at +-6), every step one fp32 operation.
 *   x      [num_rows, hidden_size] bf16, device, 16-byte aligned
 *   q      [num_rows, hidden_size / 2] bytes, device (written): element 2i in the low
 *          nibble of byte i; codes: bit 3 the sign, magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
 *   sf     [num_rows, hidden_size / 16] e4m3fn bytes, device (written)
 * hidden_size a positive multiple of 16, global_scale > 0 and finite; num_rows = 0 is a
 * no-op. Asynchronous on `stream`; INVALID_ARG for bad sizes or pointers.
 */
gbmoe_status_t moe_quant_nvfp4(int32_t num_rows, int32_t hidden_size, const void* x,
                               float global_scale, uint8_t* q, uint8_t* sf,
                               gbmoe_stream_t stream);

/*
 * moe_nvfp4_prepare_weight: rewrites one NVFP4 weight stack [rows, K] (the checkpoint
 * layout: packed codes [rows, K / 2], low nibble first, and e4m3 block scales [rows,
 * K / 16]) into the layout the NVFP4 expert GEMMs stream, as the pages' layer shuffles its
 * fp4 weights once at load time: for each tile of 128 rows and stage of 64 K values one
 * 4608-byte chunk, chunk (tile, kb) at byte (tile * K / 64 + kb) * 4608, holding
 *   bytes [h * 2048 + r * 16, +16)  the codes of row tile * 128 + r, values kb * 64 + 32 h
 *                                   .. + 31 (h = 0, 1)
 *   bytes [4096 + r * 4, +4)        that row's four block scales of the stage.
 * A permutation of bytes only. rows a positive multiple of 128, K of 64; packed, scales
 * and out 16-byte aligned device buffers; out holds moe_nvfp4_prepared_bytes(rows, K)
 * bytes (= rows * K * 9 / 16). Asynchronous on `stream`; INVALID_ARG for bad sizes or
 * pointers.
 */
size_t moe_nvfp4_prepared_bytes(int32_t rows, int32_t K);
gbmoe_status_t moe_nvfp4_prepare_weight(int32_t rows, int32_t K, const uint8_t* packed,
                                        const uint8_t* block_scale, uint8_t* out,
                                        gbmoe_stream_t stream);

/*
 * Byte offsets of the intermediate results inside a moe_forward workspace
 * (for inspection and tests). Each is valid after the call completes.
 */
typedef struct {
  size_t status;                 /* int32 device status word (see moe_get_device_status) */
  size_t topk_weights;           /* fp32 [T, top_k] */
  size_t topk_ids;               /* int32 [T, top_k] */
  size_t sorted_token_ids;       /* int32 [T*top_k + E*(bs-1)] */
  size_t expert_ids;             /* int32 [that / bs + 1] */
  size_t num_tokens_post_padded; /* int32 [1] */
  size_t act;                    /* bf16 [rows, I]: silu(gate)*up in expert order
                                    (FP8_BLOCK128: e4m3fn [rows, I], then fp32 scales
                                    [I/128][rows] at act_scale; NVFP4: f16 [rows, I], the
                                    values q * sf of the act's block quantization) */
  size_t act_scale;              /* FP8_BLOCK128 only, else 0 */
  size_t total;                  /* == moe_forward_workspace_size() */
  size_t act_shared;             /* the shared expert's act [T, I_s] in token order (bf16;
                                    NVFP4: f16 values q * sf of the quantized act); 0 when
                                    there is no shared expert */
} gbmoe_workspace_layout_t;
gbmoe_status_t moe_forward_workspace_layout(const gbmoe_config_t* cfg, int32_t max_num_tokens,
                                            gbmoe_workspace_layout_t* layout);

/*
 * moe_get_device_status: wait for `stream`, copy the int32 status word at the
 * start of `workspace` (a moe_forward or moe_align_block_size workspace) to
 * *status (GBMOE_OK or a negative gbmoe_status_t) and reset it to GBMOE_OK.
 * Returns GBMOE_ERR_CUDA if the copy fails.
 */
gbmoe_status_t moe_get_device_status(void* workspace, int32_t* status, gbmoe_stream_t stream);

/*
 * moe_forward_num_launches: number of kernels one moe_forward(cfg, num_tokens, ...)
 * enqueues (it depends on num_tokens: the small-batch routing path, split-K reduces).
 * Returns -1 for an invalid configuration.
 */
int32_t moe_forward_num_launches(const gbmoe_config_t* cfg, int32_t num_tokens);

/*
 * moe_forward_num_launches_ex: moe_forward_num_launches for a moe_forward_ex call that
 * passes the gate weight instead of router logits when from_gate_weight != 0. Batches of
 * at most 16 tokens (when num_tokens * top_k <= 2048) compute the router logits inside
 * their routing launch (the count is unchanged); larger ones add one router GEMM launch.
 * Returns -1 for an invalid configuration.
 */
int32_t moe_forward_num_launches_ex(const gbmoe_config_t* cfg, int32_t num_tokens,
                                    int32_t from_gate_weight);

/*
 * moe_selftest_bounded_wait: failure-detection self test. Enqueues one kernel whose
 * single thread waits on a shared-memory mbarrier that nothing completes, with the
 * same bounded wait the GEMM pipelines use, but giving up after timeout_us
 * (0..10^7) instead of one second; it then records GBMOE_ERR_TIMEOUT in the status
 * word of `workspace` (read it with moe_get_device_status) and exits, leaving the
 * context usable. Has no counterpart on the pages.
 */
gbmoe_status_t moe_selftest_bounded_wait(void* workspace, int32_t timeout_us,
                                         gbmoe_stream_t stream);

/*
 * ---- The decoder block around the layer: norm, paged cache, attention.
 *
 * moe_rms_norm: root-mean-square norm of each row with the residual's addition, written as
 * bf16, as the FP8 layer's quantized input, or both:
 *   h = x + residual (fp32; h = x without one), residual_out = bf16(h)
 *   y = h / sqrt(mean(h^2) + eps) * weight (fp32), y_out = bf16(y)
 *   s = max(max |y|, 1e-10) / 448 over each 128 columns, q = e4m3fn(y / s) (round to nearest
 *   even, saturating; from the fp32 y, not from its bf16 rounding). The fp32 quotient is the
 *   product with 1 / s, corrected once by what it leaves of y: where y / s lies within an fp32
 *   rounding of the border between two codes, either may come out.
 *   x             [T, H] bf16, row t at x + t * x_stride (elements)
 *   residual      [T, H] bf16, row stride residual_stride; or NULL
 *   weight        [H] bf16
 *   y             [T, H] bf16 (out) or NULL
 *   residual_out  [T, H] bf16 (out) or NULL; needs a residual; may be x's or residual's own
 *                 contiguous memory
 *   q, scale      [T, H] e4m3fn bytes and [H / 128, T] fp32, group-major as in
 *                 moe_quant_fp8_per_token_group (out); both or neither
 * At least one of y and q. H a multiple of 8 (of 128 with q), at most 32768 (else UNSUPPORTED);
 * strides multiples of 8 and >= H; bf16 pointers and q 16-byte aligned; eps >= 0. A row with a
 * NaN or an infinity gives NaN codes and values there. T = 0 is a no-op.
 */
typedef struct {
  const void* x;
  int64_t x_stride;
  const void* residual;
  int64_t residual_stride;
  const void* weight;
  float eps;
  void* y;
  void* residual_out;
  uint8_t* q;
  float* scale;
} gbmoe_rms_norm_args_t;
gbmoe_status_t moe_rms_norm(int32_t num_tokens, int32_t hidden_size,
                            const gbmoe_rms_norm_args_t* args, gbmoe_stream_t stream);

typedef enum { GBMOE_CACHE_BF16 = 0, GBMOE_CACHE_E4M3 = 1 } gbmoe_cache_type_t;

/*
 * Attention configuration of one layer.
 *  num_q_heads, num_kv_heads  query head h reads kv head h / (num_q_heads / num_kv_heads);
 *                             num_q_heads a multiple of num_kv_heads, at most 1024
 *  head_dim                   64 or 128 (else UNSUPPORTED)
 *  page_size                  tokens per page, a power of two from 8 to 1024 (else UNSUPPORTED)
 *  cache_type                 gbmoe_cache_type_t; E4M3: k = code * k_scale, v = code * v_scale
 *  causal                     !=0: a token attends no later position than its own
 *  window                     > 0: only the last `window` positions up to its own; 0 = all
 *  softmax_scale              multiplies q . k
 *  k_scale, v_scale           1 with a bf16 cache; their reciprocals are finite
 */
typedef struct {
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t cache_type;
  int32_t causal;
  int32_t window;
  float softmax_scale;
  float k_scale;
  float v_scale;
} gbmoe_attn_config_t;

/*
 * The paged cache and the sequences of one call.
 *  k_cache, v_cache  [num_pages, page_size, num_kv_heads, head_dim]: element (page, row, head, d)
 *                    at page * page_stride + row * token_stride + head * head_stride + d, the
 *                    same strides (elements, multiples of 16 bytes) for both; 16-byte aligned
 *  block_table       [num_seqs, block_table_stride] int32: entry i of a sequence is the page of
 *                    its positions [i * page_size, (i + 1) * page_size). Entries past its length
 *                    (and, for attention, wholly outside every window) are never read.
 *  cu_seqlens_q      [num_seqs + 1] int32, ascending: sequence s has the packed new tokens
 *                    [cu[s], cu[s + 1]); none is allowed
 *  kv_lens           [num_seqs] int32: positions of each sequence, its new tokens (the last
 *                    n = cu[s + 1] - cu[s] of them) among them; 0 is allowed
 * num_seqs 1..8192. The three arrays are device memory, read by the kernels: a captured graph
 * replays with their current contents. A page id outside the cache, cu_seqlens_q outside the
 * batch, a length outside the block table or a position outside cos_sin sets
 * GBMOE_ERR_DEVICE_CHECK in the device status; nothing outside the buffers is touched, and
 * the sequences concerned have unspecified outputs.
 */
typedef struct {
  void* k_cache;
  void* v_cache;
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
  int32_t num_pages;
  int32_t num_seqs;
  int32_t block_table_stride;
  const int32_t* block_table;
  const int32_t* cu_seqlens_q;
  const int32_t* kv_lens;
} gbmoe_paged_kv_t;

/*
 * moe_kv_append: rotary embedding of the new tokens' q and k, and the write of their k and v
 * into the cache. The token at index i of sequence s sits at position p = kv_lens[s] - n + i.
 * The first `rotary_dim` columns of every q and k head turn pairwise,
 *   (a, b) -> (a cos - b sin, b cos + a sin),
 * pair i being columns (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved != 0; all in
 * fp32, rounded once (E4M3: code = e4m3fn(value / scale), saturating at +-448, the quotient
 * formed as moe_rms_norm's).
 *   q, k, v     [T, heads, head_dim] bf16, token strides q_stride, k_stride, v_stride (elements,
 *               multiples of 8; heads contiguous), so that one packed projection serves
 *   cos_sin     [max_position, rotary_dim] fp32: rotary_dim / 2 cosines, then as many sines; or
 *               NULL with rotary_dim 0 (no rotation)
 *   q_out       [T, num_q_heads, head_dim] bf16 contiguous (out); may be q itself
 *   workspace   256 bytes, 256-byte aligned: the status word; or NULL (unreported)
 * rotary_dim a multiple of 16, at most head_dim. A token of no sequence is left out. T = 0 is a
 * no-op. Sequences must not share the pages that a call writes.
 */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  const float* cos_sin;
  int32_t max_position;
  int32_t rotary_dim;
  int32_t interleaved;
  void* q_out;
  void* workspace;
} gbmoe_kv_append_args_t;
gbmoe_status_t moe_kv_append(const gbmoe_attn_config_t* cfg, int32_t num_tokens,
                             const gbmoe_paged_kv_t* kv, const gbmoe_kv_append_args_t* args,
                             gbmoe_stream_t stream);

/*
 * moe_paged_attention: softmax attention of every sequence's new tokens over its pages, in one
 * call for single tokens, chunks after a context and whole prompts (kv_lens = n) alike.
 * Token i of sequence s at position p = kv_lens[s] - n + i attends the keys j with
 *   0 <= j < kv_lens[s], j <= p if causal, j > p - window if window > 0;
 *   out = sum_j softmax_j(softmax_scale q . k_j) v_j, lse = log sum_j exp(softmax_scale q . k_j).
 * A token without keys has out = 0 and lse = -inf; a row of `out` in no sequence is unspecified.
 * Scores, the softmax's maximum and sum, and the output's sums are fp32; the weights are
 * rounded for their product with v: to bf16 with a bf16 cache, to f16 with E4M3, where weights
 * below 2^-32 of the row's largest are lost (N keys: at most N * 2^-32 of that weight). With E4M3
 * q is rounded to f16 before its product with k: exact from 2^-14 to 65504 in magnitude, with
 * fewer bits below, saturating at +-65504 above. What pages hold past a sequence's length, or
 * outside every window of the call, is ignored whatever it is; v of the positions inside must be
 * finite even where a mask hides them from some of the tokens.
 *   q    [T, num_q_heads, head_dim] bf16, token stride q_stride (elements, a multiple of 8)
 *   out  [T, num_q_heads, head_dim] bf16 contiguous (out)
 *   lse  [T, num_q_heads] fp32 (out) or NULL
 * Workspace: moe_paged_attention_workspace_size(cfg) bytes (0: bad configuration), 256-byte
 * aligned, its first 1024 bytes zeroed once (and again after a GBMOE_ERR_TIMEOUT: beside the
 * status word they hold counters that every completed call leaves at zero). T = 0 is a no-op;
 * T * num_q_heads at most 2^30. The work is counted in 32 bits (else UNSUPPORTED): with P the
 * positions of a block table row (at most 2^30), one of these below 2^31 is enough,
 *   num_kv_heads * (T * group / 8 + num_seqs) * (P / 128 + 5), or, when T * group > 16 * num_seqs,
 *   num_kv_heads * (T * group / 256 + num_seqs) * (P / 128 + 5), five times that with heads of 64.
 */
size_t moe_paged_attention_workspace_size(const gbmoe_attn_config_t* cfg);
gbmoe_status_t moe_paged_attention(const gbmoe_attn_config_t* cfg, int32_t num_tokens,
                                   const gbmoe_paged_kv_t* kv, const void* q, int64_t q_stride,
                                   void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, gbmoe_stream_t stream);

/*
 * ---- The products around the layer: dense projections and experts' products by themselves.
 *
 * moe_linear: a matrix product with its epilogue,
 *   z = x @ weight^T + bias                                (fp32 sums)
 *   a = act(z); SILU_MUL: a = silu(z[:, :out_features / 2]) * z[:, out_features / 2:]
 *   out = bf16(a * row_weight[t] + residual)               (fp32, rounded once)
 * moe_grouped_linear: the same where row t of run g, offsets[g] <= t < offsets[g + 1], meets
 * weight[g] and bias[g]: the experts' products over rows that lie sorted by expert already.
 *   x             [T, in_features] bf16, or e4m3fn bytes with weight_quant FP8_BLOCK128; row t at
 *                 x + t * x_stride (elements)
 *   x_scale       FP8_BLOCK128: [in_features / 128, T] fp32, group-major, as moe_rms_norm and
 *                 moe_quant_fp8_per_token_group write it; else NULL
 *   weight        [out_features, in_features] (grouped: [num_groups, out_features, in_features])
 *                 contiguous, of x's type
 *   weight_scale  FP8_BLOCK128: [ceil(out_features / 128), in_features / 128] fp32 per group
 *                 (w = q * scale[n / 128][k / 128]); else NULL
 *   bias          [out_features] bf16 (grouped: [num_groups, out_features]) or NULL
 *   activation    gbmoe_epilogue_t. SILU_MUL takes the rows of `weight` (and the bias) as gate
 *                 [0, out_features / 2) and up behind it, as w13 lies, and has out_features / 2
 *                 output columns
 *   residual      [T, output columns] bf16, row stride residual_stride; or NULL
 *   row_weight    [T] fp32 or NULL (1)
 *   out           [T, output columns] bf16 (out), row stride out_stride; may be the residual's own
 *                 memory (the same stride), must not overlap anything else that the call reads
 *   offsets       [num_groups + 1] int32, ascending, device memory that the kernel reads: a captured
 *                 graph replays with its current contents. Empty runs are allowed; rows before
 *                 offsets[0] and from offsets[num_groups] on are left as they are.
 *   workspace     256 bytes, 256-byte aligned: the status word; or NULL: then a failed device check or a
 *                 bounded wait that ran out, which may leave rows unwritten, is reported nowhere
 * T: at most 2^22. in_features: a multiple of 8 (FP8_BLOCK128: of 128), at most 2^24. out_features: any; with SILU_MUL
 * a multiple of 32 (FP8_BLOCK128: of 256). Else UNSUPPORTED, as are NVFP4, more than 1024 groups,
 * 2^31 - 1024 or more rows of all weights together, x_stride from 2^39 on, and calls of more than 2^30
 * output tiles (of 128 columns by 16 rows). x 16-byte aligned, x_stride a multiple of 16 bytes; weight
 * 16-byte aligned; the others aligned to their elements. A run that is negative or outside [0, T]
 * sets GBMOE_ERR_DEVICE_CHECK and has no rows; runs that overlap have unspecified outputs where they
 * do, and where runs go back and come again, so that they add up to more than T rows, later ones may
 * have none. A NaN or an infinity in a row of x reaches that row alone, in a row of weight that column alone
 * (SILU_MUL: its pair's). Sums are fp32 throughout (e4m3: per block of 128 columns, then scaled and
 * added in fp32). The order of a sum goes by the call's sizes and groups, so that a row may round
 * differently in another batch; the same call gives the same bits.
 * T = 0 is a no-op.
 */
typedef enum {
  GBMOE_EPI_NONE = 0,
  GBMOE_EPI_RELU = 1,
  GBMOE_EPI_SILU = 2,
  GBMOE_EPI_GELU = 3,       /* z * (1 + erf(z / sqrt 2)) / 2 */
  GBMOE_EPI_GELU_TANH = 4,  /* z * (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
  GBMOE_EPI_SILU_MUL = 5
} gbmoe_epilogue_t;
typedef struct {
  const void* x;
  int64_t x_stride;
  const float* x_scale;
  const void* weight;
  const float* weight_scale;
  const void* bias;
  int32_t activation;
  int32_t weight_quant;  /* gbmoe_weight_quant_t */
  const void* residual;
  int64_t residual_stride;
  const float* row_weight;
  void* out;
  int64_t out_stride;
  void* workspace;
} gbmoe_linear_args_t;
gbmoe_status_t moe_linear(int32_t num_tokens, int32_t in_features, int32_t out_features,
                          const gbmoe_linear_args_t* args, gbmoe_stream_t stream);
gbmoe_status_t moe_grouped_linear(int32_t num_tokens, int32_t num_groups, int32_t in_features,
                                  int32_t out_features, const int32_t* offsets,
                                  const gbmoe_linear_args_t* args, gbmoe_stream_t stream);

/* Library version, (major << 16) | minor. */
int32_t gbmoe_version(void);

#ifdef __cplusplus
}
#endif
#endif /* GBMOE_H */
