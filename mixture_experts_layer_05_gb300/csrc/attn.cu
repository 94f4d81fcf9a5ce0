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
  return line_bound(attn_shape<AttnShapeOf<5, 5>>(a, 3, 15), a.b.T, a.b.S, cap) < 2147483647.0;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  // query rows per sequence and kv head, on average (the lengths are on the device); either
  // kernel is right for any. 32 sequences of 2200 keys, 8 kv heads of 4 query heads, 1, 4, 6 and 8
  // tokens each: 52, 61, 125, 132 us in units of 8 and 16 rows, 60, 61, 61, 62 on the tensor cores
  // (units of 256); 5 sequences of 47500 keys and 16 query heads a kv head in e4m3 73 and 88.
  const long long G = a.hq / a.hkv;
  const long long rows = (long long)a.b.T * G;
  if (rows <= 16ll * a.b.S) return launch_attn_decode(a, rows <= 8ll * a.b.S, stream);
  return launch_attn_tc(a, stream);
}

}  // namespace gbmoe
