// Index rules of the paged batch, free of CUDA so that they also compile for the host: what a
// sequence's sizes and a page id are cut to when they lie outside their buffers, and the keys
// that a new token attends.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GBMOE_HD __host__ __device__ __forceinline__
#define GBMOE_ROLLED _Pragma("unroll 1")
#else
#define GBMOE_HD inline
#define GBMOE_ROLLED
#endif

namespace gbmoe {

struct SeqInfo {
  int q0, n, L;  // first new token, new tokens, keys
};
struct KeyRange {
  int lo, hi;    // keys [lo, hi); lo >= hi: none
};

// Sequence with new tokens [q0, q1) of a batch of T, L keys, and a block table of cap positions:
// tokens outside the batch are dropped and lengths cut to [0, cap]; *bad is set for either.
GBMOE_HD SeqInfo checked_seq(int q0, int q1, int L, int T, long long cap, bool* bad) {
  SeqInfo r;
  r.q0 = q0;
  r.n = 0;
  r.L = L;
  const long long most = cap < (1ll << 30) ? cap : (1ll << 30);
  if (q0 < 0 || q1 < q0 || q1 > T) {
    *bad = true;
    r.q0 = 0;
  } else {
    r.n = q1 - q0;
  }
  if (L < 0 || L > most) {
    *bad = true;
    r.L = L < 0 ? 0 : (int)most;
  }
  return r;
}

// Keys of the sequence's new token i.
GBMOE_HD KeyRange key_range(const SeqInfo& q, int i, bool causal, int window) {
  const int pos = q.L - q.n + i;
  KeyRange r;
  r.hi = causal && pos + 1 < q.L ? pos + 1 : q.L;
  // compared before it is subtracted: pos may be below 0, window up to 2^31 - 1
  r.lo = window > 0 && pos >= window ? pos - window + 1 : 0;
  return r;
}

GBMOE_HD int checked_page(int id, int num_pages, bool* bad) {
  if ((uint32_t)id < (uint32_t)num_pages) return id;
  *bad = true;
  return 0;
}

}  // namespace gbmoe
