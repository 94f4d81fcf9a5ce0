// Device helpers of the paged batch: a sequence's checked sizes, the page of a key, and the
// sequence of a packed token.
#pragma once

#include "block.h"
#include "common.cuh"
#include "paged_checks.h"

namespace gbmoe {

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
