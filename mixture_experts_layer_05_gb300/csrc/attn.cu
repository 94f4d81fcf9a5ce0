// Paged attention: launches the kernel of the units that a batch runs in (unit_shift).
#include "attn.cuh"
#include "kernels.h"

namespace gbmoe {

cudaError_t launch_attn_decode(const AttnArgs& a, bool eight, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t stream);

namespace {
int shift_of(const AttnArgs& a) {
  return unit_shift(a.hq / a.hkv, a.hkv, a.D, a.fp8, a.b.T, a.b.S,
                    (double)a.b.table_stride * (1 << a.b.page_shift));
}
}  // namespace

size_t attn_scratch_bytes(int D) {
  return kAttnMaxCtas * (sizeof(AttnRec) + 2 * (size_t)kAttnMaxBR * (sizeof(float2) + D * 4));
}

bool attn_fits(const AttnArgs& a) { return shift_of(a) != 0; }

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  const int shift = shift_of(a);
  return shift == 8 ? launch_attn_tc(a, stream) : launch_attn_decode(a, shift == 3, stream);
}

}  // namespace gbmoe
