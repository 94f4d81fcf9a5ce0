// Shared by the kernels of the dense and grouped products (linear_stream.cu, linear_pair.cu, linear_fp8.cu):
// the line of work units, waits and copies, the activations, and the epilogue of weights on M.
//
// A unit is (group, row block, tile of features); a group's units follow one another, row blocks fastest
// within sections of `gm` blocks, so that a weight tile is read from HBM once. linear_stream.cu and
// linear_pair.cu put the weights on the MMA's M side (a TMEM lane is an output feature) and a block of at
// most `bn` rows of one group on N, so a ragged run costs no more than its rows rounded up to 16;
// linear_fp8.cu has 128 rows of one group on M.
//
// Both types have K blocks of 128 bytes (64 bf16, 128 e4m3: one swizzle row, one scale block).
// With SILU_MUL a tile of weight rows holds 16 gate rows, the 16 up rows of the same features, and
// so on, through a five-dimensional tensor map: lane l < 16 of a warp then has the gate and lane
// l + 16 the up half of one feature, and a shuffle brings them together.
#pragma once

#include "linear.h"
#include "linear_plan.h"
#include "tc.cuh"

namespace gbmoe {

constexpr int kLinWRows = 128;                  // weight rows per CTA and MMA
constexpr uint32_t kLinWBytes = kLinWRows * 128;
constexpr uint32_t kLinSmemMax = 232448;

// One launch: the call, and how it is cut.
struct LinLaunch {
  LinearArgs a;
  int bn;          // rows per block, a multiple of 16
  int n_tiles;     // feature tiles of the weights of one group
  int gm;          // row blocks walked together across the feature tiles
  int k_blocks;
  int stages;
  int tab_off;     // byte offsets in shared memory, from the aligned base: group table,
  int bar_off;     // barriers,
  int red_off;     // partial sums of a cluster (stream kernel), values on their way out (e4m3),
  int scale_off;   // row scales (e4m3),
  int half_off;    // (stream kernel, e4m3) sums of every other K block
  // stream kernel
  int cluster;     // CTAs that cut a unit's K blocks
  int rows[kLinChoices];  // weight rows per tile: the choices (the kernel picks, by its groups), largest first,
  int choices;     // and how many
  int kps;         // K blocks per stage
  int whole;       // K is whole K blocks: a box takes kps of them
};

namespace {

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z, int v, int w) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(v), "r"(w)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int x, int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int x, int y, int z, int v, int w,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(v), "r"(w),
      "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int x, int y, int z, int v,
                                                 int w) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "r"(v),
      "r"(w)
      : "memory");
}
__device__ __forceinline__ void lin_prefetch(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// One thread of a converged warp. Unlike a test of the lane it tells the compiler that there is one, so
// that the descriptors of the TMA and MMA instructions stay in uniform registers (with a test of the lane
// each TMA took 70 ns to issue, with this one a few).
__device__ __forceinline__ bool lin_elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(r));
  return r != 0;
}
// The waits. With CLUSTER they acquire at the scope of the cluster, which a phase that another CTA's
// arrivals, copies or MMAs complete needs; without, at that of the CTA.
template <bool CLUSTER>
__device__ __forceinline__ bool lin_try(uint32_t bar, uint32_t parity) {
  return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
}
// One thread's, across the cluster (wait_fast is the other).
__device__ __forceinline__ bool wait_fast_cluster(uint32_t bar, uint32_t parity,
                                                  volatile int* abort_flag, int* status) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  return wait_bounded_cluster(bar, parity, abort_flag, status);
}
// A whole warp's. Where one gives up, some lanes may still see the phase complete; all of them have to go
// the same way, to loads from TMEM and barriers that take the warp as one. (Inlined: behind a call the e4m3
// kernels' sums leave the registers, 8192 gated rows in 16 groups 236 us for 217.)
template <bool CLUSTER = false>
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         int* status) {
  if (__all_sync(0xffffffffu, lin_try<CLUSTER>(bar, parity))) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, lin_try<CLUSTER>(bar, parity))) return true;
    if ((i & 63u) == 0u) {
      if (__any_sync(0xffffffffu, *abort_flag)) return false;
      if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitTimeoutNs)) {
        *abort_flag = 1;
        record_status(status, GBMOE_ERR_TIMEOUT);
        return false;
      }
    }
  }
}
// The end of a kernel's work, by all threads: a barrier of the block or of the cluster of C CTAs, behind which
// none uses another's shared memory. Where one of them gave up, all of them stay until what is still in
// flight to or from their shared memory and TMEM (copies, MMAs, partial sums) has landed. That takes
// microseconds, and the barriers that would tell may never complete; a millisecond is far behind it.
constexpr unsigned long long kLinSettleNs = 1000000;
__device__ __noinline__ void lin_tell(int C, volatile int* abort_flag) {
  for (int r = 0; r < C; ++r)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                     mapa_shared(smem_addr(const_cast<int*>(abort_flag)), r)),
                 "r"(1)
                 : "memory");
}
__device__ __noinline__ void lin_settle(int C) {
  const unsigned long long t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < kLinSettleNs) {}
  __syncwarp();
  if (C > 1) cluster_sync();
  else __syncthreads();
}
__device__ __forceinline__ void lin_leave(int C, volatile int* abort_flag) {
  // the vote brings the warp together for the barrier, without __syncwarp's wait for its stores (96 rows of
  // 2048 to 2048 9.8 us for 9.3)
  const bool gave_up = __any_sync(0xffffffffu, *abort_flag);
  if (C > 1) {
    if (gave_up) lin_tell(C, abort_flag);
    cluster_sync();
  } else {
    __syncthreads();
  }
  if (*abort_flag) lin_settle(C);                  // the same for all threads
}
// a0 += s0 * v0, a1 += s1 * v1 (two IEEE fmas in one instruction).
__device__ __forceinline__ void fma2(float& a0, float& a1, float s0, float s1, float v0, float v1) {
  asm("{\n\t.reg .b64 a, v, s;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 s, {%2, %3};\n\t"
      "mov.b64 v, {%4, %5};\n\t"
      "fma.rn.f32x2 a, s, v, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(s0), "f"(s1), "f"(v0), "f"(v1));
}

// ---------------------------------------------------------------- units
struct LinUnit {
  int g, nt;     // group, feature tile
  int m0, n;     // first row, rows
  bool alone;    // the group's only row block: its weights have no other reader
};

// The groups of a launch, in shared memory: row blocks before each, first row, rows.
struct LinGroups {
  int* before;   // [G + 1]
  int* first;    // [G]
  int* rows;     // [G]
  int G;

  __device__ __forceinline__ LinGroups(int* tab, int groups)
      : before(tab), first(tab + groups + 1), rows(tab + 2 * groups + 1), G(groups) {}

  // By the whole block; ends with a barrier.
  __device__ void load(const LinLaunch& L) {
    const LinearArgs& a = L.a;
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
      int lo = 0, hi = a.T;
      if (a.offsets) {
        lo = a.offsets[g];
        hi = a.offsets[g + 1];
        if (lo < 0 || hi < lo || hi > a.T) {
          record_status(a.status, GBMOE_ERR_DEVICE_CHECK);
          lo = hi = 0;
        }
      }
      first[g] = lo;
      rows[g] = hi - lo;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      // Ascending runs have fewer blocks. Those that go back and come again could have so many that their
      // units pass 32 bits; they are wrong, and keep what is below.
      const int most = (a.T + L.bn - 1) / L.bn + G;
      int carry = 0;
      for (int g0 = 0; g0 < G; g0 += 32) {
        const int g = g0 + lane;
        int v = g < G ? (rows[g] + L.bn - 1) / L.bn : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += t;
        }
        if (g < G) before[g + 1] = min(carry + v, most);
        carry += __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) before[0] = 0;
    }
    __syncthreads();
  }

  __device__ __forceinline__ int units(int n_tiles) const { return before[G] * n_tiles; }

  __device__ __forceinline__ LinUnit unit(const LinLaunch& L, int n_tiles, int u) const {
    const int b = u / n_tiles;
    int g = 0, end = G;
    while (end - g > 1) {
      const int mid = (g + end) >> 1;
      if (before[mid] <= b) g = mid;
      else end = mid;
    }
    return place(L, n_tiles, u, g, before[g], before[g + 1] - before[g], first[g], rows[g]);
  }

  // Unit u of group g, whose `blocks` row blocks come after `before` others.
  __device__ __forceinline__ static LinUnit place(const LinLaunch& L, int n_tiles, int u, int g,
                                                  int before, int blocks, int first, int rows) {
    const int s0 = (u / n_tiles - before) / L.gm * L.gm;  // this section's first block
    const int sn = min(L.gm, blocks - s0);
    const int local = u - (before + s0) * n_tiles;
    LinUnit r;
    r.g = g;
    r.nt = local / sn;
    const int at = (s0 + local % sn) * L.bn;
    r.m0 = first + at;
    r.n = min(L.bn, rows - at);
    r.alone = blocks == 1;
    return r;
  }
};

// ---------------------------------------------------------------- epilogue
// The quotients by __fdividef: 2 ulp, where the result is rounded to bf16 next. A denominator past
// 2^126 gives 0, where the true value is below 1e-35.
__device__ __forceinline__ float lin_silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }
// z (1 + erf(z / sqrt 2)) / 2 = max(z, 0) - |z| q, q = erfc(|z| / sqrt 2) / 2, which does not cancel where z is
// negative as 1 + erf does. q = exp(-z^2 / 2) t P(t) with t = 1 / (1 + 0.42 |z| / sqrt 2), as in the formulas of
// Abramowitz and Stegun's 7.1.26; P is a fit of its own, of degree 7 and within 1.7e-7 of q for |z| up to 13.
// (4096 rows of 512 to 6144: 54 us, with 1 + erff 56, with erfcf 80.)
__device__ __forceinline__ float lin_gelu(float z) {
  const float s = fmaxf(-z, fminf(z, 16.f));       // |z|, where q is not 0 for positive z
  const float t = __fdividef(1.f, fmaf(0.29698485f, s, 1.f));
  float p = 0.0351963863f;
  p = fmaf(p, t, -0.160469383f);
  p = fmaf(p, t, 0.220932662f);
  p = fmaf(p, t, -0.0658207536f);
  p = fmaf(p, t, 0.134671509f);
  p = fmaf(p, t, 0.0972703174f);
  p = fmaf(p, t, 0.119808093f);
  p = fmaf(p, t, 0.118411101f);
  return fmaf(-s, __expf(-0.5f * z * z) * (t * p), fmaxf(z, 0.f));
}
template <int N, class F>
__device__ __forceinline__ void lin_each(float (&y)[N], F f) {
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = f(y[i]);
}
template <int N>
__device__ __forceinline__ void lin_activate(float (&y)[N], int act) {
  switch (act) {
    case GBMOE_EPI_RELU: lin_each(y, [](float z) { return z < 0.f ? 0.f : z; }); break;
    case GBMOE_EPI_SILU: lin_each(y, [](float z) { return lin_silu(z); }); break;
    case GBMOE_EPI_GELU:
      lin_each(y, [](float z) { return lin_gelu(z); });
      break;
    case GBMOE_EPI_GELU_TANH:                      // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
      lin_each(y, [](float z) {
        return __fdividef(z, 1.f + __expf(-1.5957691f * (z + 0.044715f * z * z * z)));
      });
      break;
    default: break;
  }
}

// What this lane stores of a unit: the column of out, and its biases.
struct LinLane {
  int f;            // output column
  bool in;          // f is one
  float bias, up_bias;

  // f0: the first output column of the warp's 32 weight rows
  template <bool GATED>
  __device__ __forceinline__ static LinLane make(const LinearArgs& a, int g, int f0) {
    LinLane r;
    const int lane = threadIdx.x & 31;
    r.f = f0 + (GATED ? lane & 15 : lane);
    r.in = r.f < a.cols;
    r.bias = r.up_bias = 0.f;
    if (a.bias && r.in) {
      const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(a.bias) + (long long)g * a.N;
      r.bias = __bfloat162float(b[r.f]);
      if (GATED) r.up_bias = __bfloat162float(b[a.cols + r.f]);
    }
    return r;
  }
};

// What the epilogue adds to COLS values of this lane: row weights and residual of rows t0 .. t0 + cnt.
template <bool GATED, int COLS>
struct LinExtra {
  float rw[COLS];
  __nv_bfloat16 res[COLS];

  // Unconditional loads (rows past the last repeat it), so that they fly together; called early, they
  // fly under the products.
  __device__ __forceinline__ void fetch(const LinearArgs& a, const LinLane& l, int t0, int cnt) {
    if (GATED && (threadIdx.x & 16)) {
      t0 += COLS;
      cnt -= COLS;
    }
    if (!l.in || cnt <= 0) return;
    if (a.row_weight) {
#pragma unroll
      for (int i = 0; i < COLS; ++i) rw[i] = __ldg(a.row_weight + t0 + min(i, cnt - 1));
    }
    if (a.residual) {
      const __nv_bfloat16* r =
          static_cast<const __nv_bfloat16*>(a.residual) + (long long)t0 * a.residual_stride + l.f;
#pragma unroll
      for (int i = 0; i < COLS; ++i) res[i] = r[min(i, cnt - 1) * a.residual_stride];
    }
  }
};

// 2 COLS (GATED) or COLS values per lane: the sums of the warp's weight rows for rows t0 .. t0 + cnt
// of x, cnt <= the number of values. With GATED lanes l and l + 16 swap halves: the lower keep the
// first half of the columns, the upper the second.
template <bool GATED, int COLS>
__device__ __forceinline__ void lin_store(const LinearArgs& a, const LinLane& l, int t0, int cnt,
                                          float (&v)[GATED ? 2 * COLS : COLS],
                                          const LinExtra<GATED, COLS>& x) {
  float y[COLS];
  if (GATED) {
    const bool upper = (threadIdx.x & 16) != 0;
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + COLS], 16);
      const float gate = (upper ? other : v[i]) + l.bias;
      const float up = (upper ? v[i + COLS] : other) + l.up_bias;
      y[i] = lin_silu(gate) * up;
    }
    if (upper) {
      t0 += COLS;
      cnt -= COLS;
    }
  } else {
#pragma unroll
    for (int i = 0; i < COLS; ++i) y[i] = v[i] + l.bias;
    lin_activate(y, a.act);
  }
  if (!l.in || cnt <= 0) return;
  if (a.row_weight) {
#pragma unroll
    for (int i = 0; i < COLS; ++i) y[i] *= x.rw[i];
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < COLS; ++i) y[i] += __bfloat162float(x.res[i]);
  }
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + (long long)t0 * a.out_stride + l.f;
#pragma unroll
  for (int i = 0; i < COLS; ++i)
    if (i < cnt) o[i * a.out_stride] = __float2bfloat16_rn(y[i]);
}

}  // namespace

// Tensor maps of a call: boxes of 128 bytes of so many rows, at (element, row, 0); or with kps > 0, for
// which K has to be whole K blocks (lin_whole), of kps K blocks at (0, row, K block). x:
inline bool lin_whole(const LinearArgs& a) { return a.K % (a.fp8 ? 128 : 64) == 0; }
bool lin_map_x(const LinearArgs& a, int rows, int kps, CUtensorMap* x);
// the weights as plain rows;
bool lin_map_rows(const LinearArgs& a, int rows, int kps, CUtensorMap* w);
// or, with SILU_MUL, in tiles of 16 gate rows, their 16 up rows, and so on: (element, 0, 2 group,
// block of 16 features, 0), or (0, 0, 2 group, block, K block).
bool lin_map_tiles(const LinearArgs& a, int rows, int kps, CUtensorMap* w);
// Clusters of `size` CTAs of the stream kernel that the device holds (0: an error).
int linear_stream_room(const LinearArgs& a, int bn, int size);
cudaError_t launch_linear_stream(LinLaunch L, long long max_units, cudaStream_t stream);
cudaError_t launch_linear_pair(LinLaunch L, long long max_units, cudaStream_t stream);
cudaError_t launch_linear_fp8(LinLaunch L, long long max_units, cudaStream_t stream);

}  // namespace gbmoe
