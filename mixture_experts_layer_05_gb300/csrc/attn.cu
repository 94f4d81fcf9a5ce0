// Paged attention: which kernel a batch runs on.
#include "attn.cuh"
#include "kernels.h"

namespace gbmoe {

cudaError_t launch_attn_decode(const AttnArgs& a, bool eight, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t stream);

size_t attn_scratch_bytes(int D) {
  return kAttnMaxCtas * (sizeof(AttnRec) + 2 * (size_t)kAttnMaxBR * (sizeof(float2) + D * 4));
}

bool attn_fits(const AttnArgs& a) {
  const double cap = (double)a.b.table_stride * (1 << a.b.page_shift);
  // units of 8 rows and the widest unit's extra cost: no launch has a longer line
  return line_bound(attn_shape(a, 3, 4), a.b.T, a.b.S, cap) < 2147483647.0;
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
