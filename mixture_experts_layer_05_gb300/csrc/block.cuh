// Device helpers of the paged batch: a sequence's checked sizes, the page of a key, and the
// sequence of a packed token.
#pragma once

#include <cuda_fp8.h>

#include "block.h"
#include "common.cuh"
#include "paged_checks.h"

namespace gbmoe {

// v / s from inv = 1 / s, for e4m3: the product, corrected by what it leaves of v (Newton's step for
// the quotient), so that a value near the border of two codes falls where the quotient falls.
// ANY: v may be far beyond 448 s or infinite; a product that saturates stays as it is.
template <bool ANY>
__device__ __forceinline__ float divided(float v, float s, float inv) {
  const float q = v * inv;
  return !ANY || fabsf(q) < 1024.f ? fmaf(fmaf(-q, s, v), inv, q) : q;
}
// Four e4m3 bytes of (a, b, c, d) / s, a in the lowest byte. Divisions proper bound the norm's
// 8-bit output (76 us for 8192 x 7168 where HBM needs 27).
template <bool ANY>
__device__ __forceinline__ uint32_t e4m3x4_divided(float a, float b, float c, float d, float s,
                                                   float inv) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
      make_float2(divided<ANY>(a, s, inv), divided<ANY>(b, s, inv)), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
      make_float2(divided<ANY>(c, s, inv), divided<ANY>(d, s, inv)), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Sizes of sequence s, cut to what can be addressed; what was outside is recorded.
__device__ __forceinline__ SeqInfo seq_info(const PagedBatch& b, int s) {
  bool bad = false;
  const SeqInfo r = checked_seq(b.cu[s], b.cu[s + 1], b.kv_lens[s], b.T,
                                (long long)b.table_stride << b.page_shift, &bad);
  if (bad) record_status(b.status, GBMOE_ERR_DEVICE_CHECK);
  return r;
}

// The page of key j of sequence s; a page id outside the cache is recorded and gives page 0.
__device__ __forceinline__ int page_of(const PagedBatch& b, int s, int j) {
  bool bad = false;
  const int p = checked_page(__ldg(b.table + (size_t)s * b.table_stride + (j >> b.page_shift)),
                             b.num_pages, &bad);
  if (bad) record_status(b.status, GBMOE_ERR_DEVICE_CHECK);
  return p;
}

// The sequence that packed token t belongs to (the whole warp calls it): the last s with
// cu[s] <= t, by a 32-way search whose steps are one load per lane; -1 when t lies outside
// every sequence.
__device__ __forceinline__ int find_seq_warp(const PagedBatch& b, int t, int lane) {
  int lo = 0, count = b.S + 1;  // candidates cu[lo .. lo + count)
  while (true) {
    const int step = (count + 31) / 32;
    const int i = lane * step;
    const bool le = i < count && b.cu[lo + i] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) return -1;
    const int last = 31 - __clz(m);
    lo += last * step;
    if (step == 1) break;
    count = min(step, count - last * step);
  }
  return lo < b.S ? lo : -1;
}

}  // namespace gbmoe
