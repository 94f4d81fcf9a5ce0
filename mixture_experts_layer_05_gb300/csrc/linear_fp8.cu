// moe_linear / moe_grouped_linear with e4m3 operands for many rows per group.
//
// Every K block of 128 has its own scales, so its product is formed by itself in TMEM (4 MMAs of K = 32)
// and promoted into fp32 registers, while the next K block's runs into the other of two buffers. Here
// the rows of x are on the MMA's M side: a TMEM lane is a row, whose scale is one register, and the
// weights' scale is the same for 128 columns, so that promoting costs one fma a value. (With the
// weights on M, as the other kernels have them, the rows' scales change from column to column, and
// reading them takes shared memory's time from the operands.) For the same reason one CTA works
// by itself: the round trip of a TMEM buffer, MMA to registers to MMA, is on the critical path, and
// with pairs of CTAs it crosses SMs (measured: 674 us for 8192 rows of 7168 to 4096 columns).
//
// Unit: 128 rows of one group by 256 weight rows (SILU_MUL: 128 gate rows and their up rows).
// Warps: 0 TMA, 1 TMEM and MMA, 2..9 epilogue: the two warps of a TMEM lane quarter take 128 columns
// each, of which every thread keeps the running sums of its row; the next 8 columns are on their
// way from TMEM while 8 are added.
#include "linear.cuh"

namespace gbmoe {
namespace {

constexpr int kBM = 128, kBN = 256;
constexpr int kStages = 4;
constexpr int kEpiWarps = 8;
constexpr int kCols = 128;                       // accumulator columns of an epilogue thread
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kABytes = kBM * 128, kBBytes = kBN * 128, kStageBytes = kABytes + kBBytes;
constexpr uint32_t kTmemCols = 512, kStride = 256;
constexpr int kAhead = 2;                        // K blocks that the scales' loads run ahead

// 32 lanes x 8 consecutive fp32 columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld8(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7])::"memory");
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    linear_fp8_kernel(const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ LinLaunch L) {
  constexpr int kTileCols = GATED ? 128 : 256;     // output columns per unit
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const LinearArgs& a = L.a;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch(&tm_w);
    tma_prefetch(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  LinGroups groups(reinterpret_cast<int*>(smem + L.tab_off), a.G);
  groups.load(L);                                  // ends with a barrier of the block
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = groups.units(L);
  const int KB = L.k_blocks;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const LinUnit w = groups.unit(L, u);
        const int row = w.g * a.N + w.nt * kTileCols;
        const int row1 = row + (GATED ? a.cols : 128);
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_fast(empty_bar(s), ph, abort_flag, a.status)) {
            ok = false;
            break;
          }
          const uint32_t sa = base + s * kStageBytes;
          mbar_expect_tx(full_bar(s), kStageBytes);
          tma_load_2d(sa, &tm_x, full_bar(s), kb * 128, w.m0);
          tma_load_2d(sa + kABytes, &tm_w, full_bar(s), kb * 128, row);
          tma_load_2d(sa + kABytes + kBBytes / 2, &tm_w, full_bar(s), kb * 128, row1);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(kBM, kBN);
      int s = 0, buf = 0;
      uint32_t ph = 0, tph = 1;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_fast(tempty_bar(buf), tph, abort_flag, a.status) ||
              !wait_fast(full_bar(s), ph, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + s * kStageBytes;
          const uint64_t da = sdesc_sw128(sa), db = sdesc_sw128(sa + kABytes);
          const uint32_t d = tmem_base + buf * kStride;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_e4m3(d, sdesc_advance(da, kk * 32), sdesc_advance(db, kk * 32), idesc, kk != 0);
          mma_commit(tfull_bar(buf));
          mma_commit(empty_bar(s));
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
          buf ^= 1;
          if (buf == 0) tph ^= 1u;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;                  // rows [32 quarter, + 32) of the block
    const int part = (warp - 2) >> 2;              // which half of the accumulator
    const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const int r = quarter * 32 + lane;
    const int wblocks = (a.N + 127) >> 7;
    int buf = 0;
    uint32_t tph = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const LinUnit w = groups.unit(L, u);
      // this thread's columns: SILU_MUL gate [64 part, + 64) and up [128 + 64 part, + 64), else
      // [128 part, + 128)
      const int f0 = w.nt * kTileCols + part * (kTileCols / 2);
      const float* w0 = a.w_scale + ((long long)w.g * wblocks + min(f0 >> 7, wblocks - 1)) * KB;
      const float* w1 = GATED ? w0 + (long long)(a.cols >> 7) * KB : w0;
      const bool in = r < w.n;
      const float* xs = a.x_scale + w.m0 + (in ? r : 0);
      float acc[kCols], sx[kAhead], s0[kAhead], s1[kAhead];
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
      auto fetch = [&](int kb, int i) {
        if (kb >= KB) return;
        sx[i] = __ldg(xs + (long long)kb * a.T);
        s0[i] = __ldg(w0 + kb);
        if (GATED) s1[i] = __ldg(w1 + kb);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i, i);
      for (int kb0 = 0; ok && kb0 < KB; kb0 += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int kb = kb0 + i;
          if (kb >= KB) break;
          const float c0 = sx[i] * s0[i], c1 = GATED ? sx[i] * s1[i] : c0;
          fetch(kb + kAhead, i);
          if (!wait_fast(tfull_bar(buf), tph, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tb = lanes + buf * kStride;
          auto col = [&](int c) {
            return GATED ? (c < 8 ? 64 * part + 8 * c : 64 + 64 * part + 8 * c)
                         : 128 * part + 8 * c;
          };
          uint32_t v[2][8];
          tmem_ld8(tb + col(0), v[0]);
          tmem_wait_ld8(v[0]);
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c) {
            if (c + 1 < kCols / 8) tmem_ld8(tb + col(c + 1), v[(c + 1) & 1]);
            const float sc = GATED && c >= 8 ? c1 : c0;
#pragma unroll
            for (int q = 0; q < 8; q += 2)
              fma2(acc[8 * c + q], acc[8 * c + q + 1], sc, sc, __uint_as_float(v[c & 1][q]),
                   __uint_as_float(v[c & 1][q + 1]));
            if (c + 1 < kCols / 8) tmem_wait_ld8(v[(c + 1) & 1]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty_bar(buf));
          buf ^= 1;
          if (buf == 0) tph ^= 1u;
        }
      }
      if (!ok) break;
      if (in) lin_store_row<GATED>(a, w.g, w.m0 + r, f0, acc);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool GATED>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& x, const LinLaunch& L, int units,
                   size_t smem, cudaStream_t stream) {
  auto kernel = linear_fp8_kernel<GATED>;
  static bool ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e == cudaSuccess ? cudaErrorInvalidDevice : e;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmemMax);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  const int grid = units < num_sms() ? units : num_sms();
  kernel<<<grid, kThreads, smem, stream>>>(w, x, L);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_fp8(LinLaunch L, int max_units, cudaStream_t stream) {
  const LinearArgs& a = L.a;
  if (!a.fp8 || L.bn != kBM) return cudaErrorInvalidValue;
  L.stages = kStages;
  L.bar_off = kStages * kStageBytes;
  const uint32_t bars = (2 * kStages + 4) * 8 + 16;
  L.tab_off = L.bar_off + bars;
  CUtensorMap w, x;
  if (!lin_map_rows(a, &w, &x, kBM)) return cudaErrorInvalidValue;
  const size_t smem = L.tab_off + 4 * (3 * a.G + 1) + 1024;
  return a.act == GBMOE_EPI_SILU_MUL ? launch<true>(w, x, L, max_units, smem, stream)
                                     : launch<false>(w, x, L, max_units, smem, stream);
}

}  // namespace gbmoe
