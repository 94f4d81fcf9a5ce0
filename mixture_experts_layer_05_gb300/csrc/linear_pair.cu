// moe_linear / moe_grouped_linear for many rows per group: bound by the tensor cores.
//
// Clusters of two CTAs run M = 256 MMAs (tcgen05.mma.cta_group::2): each CTA stages its own 128 weight
// rows and half of the block's rows of x, which is 64 bytes of operands per clock and SM at full rate,
// where an SM by itself would need 96. The block's rows are N, at most 256. Persistent: a cluster
// walks the units, and two TMEM accumulators let the epilogue of one unit run under the products of
// the next. (e4m3 operands have a kernel of their own, linear_fp8.cu.)
//
// 8192 rows of 4096 to 6144 columns: 217 us in a short run (1.9 PFLOP/s, cuBLAS's burst), 249 in long ones
// under the power cap (1.66, cuBLAS's sustained rate 1.69). Below 128 rows a unit the two copies of a K
// block, some 140 ns of the issuing thread, are what holds. (Two K blocks a stage: 235 us for 217, and 19.4
// for 16.6 with 512 rows of 4096 to 4096.)
//
// Warps: 0 TMA, 1 TMEM and MMA (leader), 2..9 epilogue, two to a TMEM lane quarter.
#include "linear.cuh"

namespace gbmoe {
namespace {

constexpr int kMaxBn = 256;
constexpr int kMaxStages = 10;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kStride = 256;                // TMEM columns of an accumulator

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kBars = 2 * kMaxStages + 4;

// The weights, and x in boxes of bn / 2 and of kFewRows rows.
constexpr int kFewRows = 32;
struct Maps {
  CUtensorMap w, x, x_few;
};

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ LinLaunch L) {
  constexpr int kTileCols = GATED ? 64 : 128;      // output columns per CTA and unit
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const LinearArgs& a = L.a;
  const int stages = L.stages;
  const uint32_t stage_bytes = kLinWBytes + (uint32_t)(L.bn / 2) * 128;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kMaxStages + 2 + b); };

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch(&maps.w);
    tma_prefetch(&maps.x);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  LinGroups groups(reinterpret_cast<int*>(smem + L.tab_off), a.G);
  groups.load(L);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t leader_full0 = mapa_shared(full_bar(0), 0);
  const uint32_t leader_tempty0 = mapa_shared(tempty_bar(0), 0);
  const int units = groups.units(L.n_tiles);
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  // in registers: behind an asm statement that touches memory, the launch's values are loaded again
  const int KB = L.k_blocks, out_features = a.N, half_bn = L.bn / 2;
  const bool grouped = a.offsets != nullptr;
  int* const status = a.status;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lin_elect()) {
      int s = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int u = first; ok && u < units; u += step) {
        const LinUnit w = groups.unit(L, L.n_tiles, u);
        const int half = ((w.n + 15) & ~15) / 2;
        const int x_row = w.m0 + rank * half;
        const int tile = w.nt * 2 + rank, w_row = w.g * out_features + tile * kTileCols;
        const bool few = grouped && half <= kFewRows && half_bn > kFewRows;
        const CUtensorMap* tx = few ? &maps.x_few : &maps.x;
        const int xr = few ? kFewRows : half_bn;
        const uint32_t bytes = 2u * (kLinWBytes + (uint32_t)xr * 128);   // both CTAs'
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_fast_cluster(empty_bar(s), ph, abort_flag, status)) {
            ok = false;
            break;
          }
          if (leader) mbar_expect_tx(full_bar(s), bytes);
          const uint32_t fb = leader_full0 + 8u * s, sw = base + s * stage_bytes;
          if (GATED)
            tma_load_5d_pair(sw, &maps.w, fb, kb * kGemmBK, 0, 2 * w.g, tile * (kTileCols / 16), 0);
          else
            tma_load_3d_pair(sw, &maps.w, fb, kb * kGemmBK, w_row, 0);
          tma_load_3d_pair(sw + kLinWBytes, tx, fb, kb * kGemmBK, x_row, 0);
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (leader && lin_elect()) {
      int s = 0, buf = 0;
      uint32_t ph = 0, tph = 1;
      bool ok = true;
      for (int u = first; ok && u < units; u += step) {
        const LinUnit w = groups.unit(L, L.n_tiles, u);
        const int n = (w.n + 15) & ~15;
        const uint32_t idesc = idesc_bf16(256, n);
        for (int kb = 0; kb < KB; ++kb) {
          if ((kb == 0 && !wait_fast_cluster(tempty_bar(buf), tph, abort_flag, status)) ||
              !wait_fast_cluster(full_bar(s), ph, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sw = base + s * stage_bytes;
          const uint64_t dw = sdesc_sw128(sw), dx = sdesc_sw128(sw + kLinWBytes);
          const uint32_t d = tmem_base + buf * kStride;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_pair(d, sdesc_advance(dw, kk * 32), sdesc_advance(dx, kk * 32), idesc,
                          kb != 0 || kk != 0 ? 1u : 0u);
          mma_commit_pair(empty_bar(s));
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
          if (kb == KB - 1) {
            mma_commit_pair(tfull_bar(buf));
            buf ^= 1;
            if (buf == 0) tph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;                  // TMEM lanes [32 quarter, + 32)
    const int part = (warp - 2) >> 2;              // which of the quarter's warps
    const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16);
    int buf = 0;
    uint32_t tph = 0;
    for (int u = first; u < units; u += step) {
      const LinUnit w = groups.unit(L, L.n_tiles, u);
      const LinLane l = LinLane::make<GATED>(
          a, w.g, (w.nt * 2 + rank) * kTileCols + quarter * (kTileCols / 4));
      // the first run of columns comes under the products, and the others' residual to L2
      constexpr int kStore = GATED ? 16 : 32;
      LinExtra<GATED, kStore> extra;
      extra.fetch(a, l, w.m0 + part * 32, w.n - part * 32);
      if (a.residual && l.in)
        for (int at = part * 32 + 64; at < w.n; at += 64)
          for (int i = 0; i < 32 && at + i < w.n; ++i)
            lin_prefetch(static_cast<const __nv_bfloat16*>(a.residual) +
                         (long long)(w.m0 + at + i) * a.residual_stride + l.f);
      if (!lin_wait<true>(tfull_bar(buf), tph, abort_flag, status)) break;
      tc_fence_after();
#pragma unroll 1
      for (int at = part * 32; at < w.n; at += 64) {
        uint32_t t[32];
        float v[32];
        tmem_ld32(lanes + buf * kStride + at, t);
        tmem_wait_ld(t);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(t[i]);
        if (at >= 64) extra.fetch(a, l, w.m0 + at, w.n - at);
        lin_store<GATED, kStore>(a, l, w.m0 + at, w.n - at, v, extra);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty0 + 8u * buf);
      buf ^= 1;
      if (buf == 0) tph ^= 1u;
    }
  }

  tc_fence_before();
  lin_leave(2, abort_flag);     // no CTA leaves while its peer may still signal or read it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <bool GATED>
cudaError_t launch(const Maps& maps, const LinLaunch& L, long long units,
                   size_t smem, cudaStream_t stream) {
  auto kernel = linear_pair_kernel<GATED>;
  static bool ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e == cudaSuccess ? cudaErrorInvalidDevice : e;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmemMax);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  const int most = num_sms() / 2, clusters = units < most ? (int)units : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, L);
}

}  // namespace

cudaError_t launch_linear_pair(LinLaunch L, long long max_units, cudaStream_t stream) {
  const LinearArgs& a = L.a;
  if (a.fp8 || L.bn < 32 || L.bn > kMaxBn || L.bn % 32) return cudaErrorInvalidValue;
  const uint32_t stage = kLinWBytes + L.bn / 2 * 128;
  const uint32_t tab = (4u * (3 * a.G + 1) + 15) & ~15u, bars = kBars * 8 + 16;
  const uint32_t rest = tab + bars + 1024;
  int stages = (int)((kLinSmemMax - rest) / stage);
  if (stages > kMaxStages) stages = kMaxStages;
  L.stages = stages;
  L.bar_off = stages * stage;
  L.tab_off = L.bar_off + bars;
  Maps maps;
  if (!lin_map_tiles(a, kLinWRows, 0, &maps.w) || !lin_map_x(a, L.bn / 2, 0, &maps.x) ||
      (a.offsets && !lin_map_x(a, kFewRows, 0, &maps.x_few)))
    return cudaErrorInvalidValue;
  const size_t smem = stages * stage + rest;
  return a.act == GBMOE_EPI_SILU_MUL ? launch<true>(maps, L, max_units, smem, stream)
                                     : launch<false>(maps, L, max_units, smem, stream);
}

}  // namespace gbmoe
