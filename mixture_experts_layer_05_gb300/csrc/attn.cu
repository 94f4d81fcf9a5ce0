// Paged attention: which kernel a batch runs on.
#include "attn.cuh"
#include "kernels.h"

namespace gbmoe {

cudaError_t launch_attn_decode(const AttnArgs& a, bool eight, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t stream);

size_t attn_scratch_bytes(int D) {
  return kAttnMaxCtas * (sizeof(AttnRec) + 2 * (size_t)kAttnMaxBR * (sizeof(float2) + D * 4));
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  // query rows per sequence and kv head, on average (the lengths are on the device); either
  // kernel is right for any
  const long long G = a.hq / a.hkv;
  const long long rows = (long long)a.b.T * G;
  if (rows <= 16ll * a.b.S) return launch_attn_decode(a, rows <= 8ll * a.b.S, stream);
  return launch_attn_tc(a, stream);
}

}  // namespace gbmoe
