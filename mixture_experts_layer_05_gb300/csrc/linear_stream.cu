// moe_linear / moe_grouped_linear for few rows per group: bound by reading the weights.
//
// A cluster of C CTAs takes a unit (128 weight rows by at most bn rows of x) and cuts its K blocks into C
// ranges, so that even a small layer keeps every SM reading. Each CTA streams its range through a ring
// of TMA stages into one TMEM accumulator (tcgen05.mma, M = 128, N = the rows rounded up to 16). The C
// partial sums are joined through distributed shared memory: each CTA sends the columns that CTA d
// finishes to d, which adds them in the order of the ranges and runs the epilogue, so the result does
// not depend on timing, and nothing is kept in a workspace between calls.
//
// Warps: 0 TMA, 1 TMEM and MMA, 2..5 epilogue (one TMEM lane quarter each), 6 (e4m3) scales. e4m3
// products are promoted to fp32 with their scales K block by K block, as the FP8 layer's are.
#include "linear.cuh"

namespace gbmoe {
namespace {

constexpr int kMaxBn = 128;
constexpr int kMaxCluster = 8;
constexpr int kMaxStages = 12;
constexpr uint32_t kTmemCols = 512;
constexpr int kEpiWarps = 4;
constexpr int kBufsMax = 32;                     // K block buffers (e4m3): 512 / 16

constexpr int threads_of(bool fp8) { return 64 + 32 * kEpiWarps + (fp8 ? 32 : 0); }
// barriers: full, empty per stage; tfull, tempty per TMEM buffer; red full, red empty; scale full,
// empty per slot
constexpr int kBars = 2 * kMaxStages + 2 * kBufsMax + 2 + 2 * kLinScaleSlots;

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <bool FP8, bool GATED>
__global__ void __launch_bounds__(threads_of(FP8), 1)
    linear_stream_kernel(const __grid_constant__ CUtensorMap tm_w,
                         const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ LinLaunch L, const int C) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const LinearArgs& a = L.a;
  const int bn = L.bn, stages = L.stages;
  const uint32_t stage_bytes = kLinWBytes + (uint32_t)bn * 128;
  float* red = reinterpret_cast<float*>(smem + L.red_off);
  float* scales = reinterpret_cast<float*>(smem + L.scale_off);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kMaxStages + kBufsMax + b); };
  const uint32_t rfull_bar = bar0 + 8u * (2 * kMaxStages + 2 * kBufsMax);
  const uint32_t rempty_bar = rfull_bar + 8u;
  const uint32_t sfull0 = rempty_bar + 8u, sempty0 = sfull0 + 8u * kLinScaleSlots;
  // TMEM buffers: two accumulators, or as many K block products as fit
  uint32_t stride = 16;
  while ((int)stride < bn) stride *= 2;
  const int bufs = FP8 ? (int)(kTmemCols / stride) : 2;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < bufs; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), kEpiWarps);
    }
    mbar_init(rfull_bar, kEpiWarps * C);
    mbar_init(rempty_bar, kEpiWarps * C);
    for (int s = 0; s < kLinScaleSlots; ++s) {
      mbar_init(sfull0 + 8u * s, 1);
      mbar_init(sempty0 + 8u * s, kEpiWarps);
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
  LinGroups groups(reinterpret_cast<int*>(smem + L.tab_off), a.G);
  groups.load(L);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = groups.units(L);
  const int first = blockIdx.x / C, step = gridDim.x / C;
  const int kb0 = (int)((long long)rank * L.k_blocks / C);
  const int kb1 = (int)((long long)(rank + 1) * L.k_blocks / C);
  constexpr int kTileCols = GATED ? 64 : 128;      // output columns per unit

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t policy = l2_evict_first_policy();
      constexpr int kStepElems = FP8 ? 128 : 64;
      uint32_t it = 0;
      int s = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int u = first; ok && u < units; u += step) {
        const LinUnit w = groups.unit(L, u);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          if (!wait_fast(empty_bar(s), ph, abort_flag, a.status)) {
            ok = false;
            break;
          }
          const uint32_t sw = base + s * stage_bytes;
          mbar_expect_tx(full_bar(s), stage_bytes);
          // weights that no other unit reads go first from L2
          if (GATED) {
            const int fb = w.nt * (kTileCols / 16);
            if (w.alone)
              tma_load_5d_hint(sw, &tm_w, full_bar(s), kb * kStepElems, 0, 0, fb, w.g, policy);
            else
              tma_load_5d(sw, &tm_w, full_bar(s), kb * kStepElems, 0, 0, fb, w.g);
          } else {
            const int row = w.g * a.N + w.nt * kTileCols;
            if (w.alone)
              tma_load_2d_hint(sw, &tm_w, full_bar(s), kb * kStepElems, row, policy);
            else
              tma_load_2d(sw, &tm_w, full_bar(s), kb * kStepElems, row);
          }
          tma_load_2d(sw + kLinWBytes, &tm_x, full_bar(s), kb * kStepElems, w.m0);
          if (++s == stages) {
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
      int s = 0, buf = 0;
      uint32_t ph = 0, tph = 1;
      bool ok = true;
      for (int u = first; ok && u < units; u += step) {
        const LinUnit w = groups.unit(L, u);
        const int n = (w.n + 15) & ~15;
        const uint32_t idesc = FP8 ? idesc_e4m3(128, n) : idesc_bf16(128, n);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (FP8 || kb == kb0) {
            if (!wait_fast(tempty_bar(buf), tph, abort_flag, a.status)) {
              ok = false;
              break;
            }
          }
          if (!wait_fast(full_bar(s), ph, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sw = base + s * stage_bytes;
          const uint64_t dw = sdesc_sw128(sw), dx = sdesc_sw128(sw + kLinWBytes);
          const uint32_t d = tmem_base + buf * stride;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t more = (FP8 ? kk != 0 : (kb != kb0 || kk != 0)) ? 1u : 0u;
            if (FP8) mma_e4m3(d, sdesc_advance(dw, kk * 32), sdesc_advance(dx, kk * 32), idesc, more);
            else mma_bf16(d, sdesc_advance(dw, kk * 32), sdesc_advance(dx, kk * 32), idesc, more);
          }
          mma_commit(empty_bar(s));
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
          if (FP8 || kb == kb1 - 1) {
            mma_commit(tfull_bar(buf));
            if (++buf == bufs) {
              buf = 0;
              tph ^= 1u;
            }
          }
        }
      }
    }
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const int row = quarter * 32 + lane;
    int buf = 0, slot = 0;
    uint32_t tph = 0, sph = 0, rph = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      const LinUnit w = groups.unit(L, u);
      const LinLane l = LinLane::make<GATED>(a, w.g, w.nt * kTileCols + quarter * (kTileCols / 4));
      float acc[FP8 ? kMaxBn : 16];
      if (FP8) {
#pragma unroll
        for (int i = 0; i < kMaxBn; ++i) acc[i] = 0.f;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_fast(sfull0 + 8u * slot, sph, abort_flag, a.status) ||
              !wait_fast(tfull_bar(buf), tph, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float* sc = scales + slot * bn * (GATED ? 2 : 1);
#pragma unroll
          for (int c = 0; c < kMaxBn / 16; ++c)
            if (c * 16 < w.n)
              lin_promote16<GATED>(acc + (FP8 ? 16 * c : 0), lanes + buf * stride, sc, 16 * c, lane >> 4);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(tempty_bar(buf));
            mbar_arrive(sempty0 + 8u * slot);
          }
          if (++buf == bufs) {
            buf = 0;
            tph ^= 1u;
          }
          if (++slot == kLinScaleSlots) {
            slot = 0;
            sph ^= 1u;
          }
        }
      } else if (!wait_fast(tfull_bar(buf), tph, abort_flag, a.status)) {
        ok = false;
      }
      if (!ok) break;
      tc_fence_after();
      // C > 1: this CTA's sums of columns [d * per, (d + 1) * per) go to CTA d
      const int per = (w.n + C - 1) / C;
      if (C > 1 && u != first) {
        if (!wait_bounded_cluster(rempty_bar, rph ^ 1u, abort_flag, a.status)) {
          ok = false;
          break;
        }
      }
#pragma unroll
      for (int c = 0; c < kMaxBn / 16; ++c) {
        if (c * 16 >= w.n) break;
        float v[16];
        if (FP8) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = acc[FP8 ? 16 * c + i : 0];
        } else {
          uint32_t t[16];
          tmem_ld16(lanes + buf * stride + 16 * c, t);
          tmem_wait_ld16(t);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(t[i]);
        }
        if (C == 1) {
          lin_store<GATED, GATED ? 8 : 16>(a, l, w.m0 + 16 * c, w.n - 16 * c, v);
        } else {
          int d = 16 * c / per, at = 16 * c - d * per;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (16 * c + i < w.n) {
              st_cluster(mapa_shared(smem_addr(red + (rank * per + at) * kLinWRows + row), d), v[i]);
              if (++at == per) {
                at = 0;
                ++d;
              }
            }
          }
        }
      }
      if (!FP8) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(buf));
        if (++buf == bufs) {
          buf = 0;
          tph ^= 1u;
        }
      }
      if (C > 1) {
        __syncwarp();
        if (lane < C) mbar_arrive_cluster(mapa_shared(rfull_bar, lane));
        if (!wait_bounded_cluster(rfull_bar, rph, abort_flag, a.status)) {
          ok = false;
          break;
        }
        const int mine = min(per, w.n - rank * per);
        for (int c0 = 0; c0 < mine; c0 += 16) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
          for (int s = 0; s < C; ++s) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c0 + i < mine) v[i] += red[(s * per + c0 + i) * kLinWRows + row];
          }
          lin_store<GATED, GATED ? 8 : 16>(a, l, w.m0 + rank * per + c0, mine - c0, v);
        }
        __syncwarp();
        if (lane < C) mbar_arrive_cluster(mapa_shared(rempty_bar, lane));
        rph ^= 1u;
      }
    }
  } else if (FP8) {
    // ------------------------------------------------------------ scales
    uint32_t it = 0;
    for (int u = first; u < units; u += step) {
      const LinUnit w = groups.unit(L, u);
      if (!LinScales<GATED, kMaxBn>::unit(L, w, w.nt * kTileCols, kb0, kb1, scales,
                                          bn * (GATED ? 2 : 1), sfull0, sempty0, it, abort_flag))
        break;
    }
  }

  tc_fence_before();
  cluster_sync();               // no CTA leaves while another may still write to it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool FP8, bool GATED>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& x, const LinLaunch& L, int C, int units,
                   size_t smem, cudaStream_t stream) {
  auto kernel = linear_stream_kernel<FP8, GATED>;
  // CTAs that the device holds of each cluster size, found once per device
  static int room[64][kMaxCluster + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e == cudaSuccess ? cudaErrorInvalidDevice : e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads_of(FP8));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!room[dev][C]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmemMax);
    if (e != cudaSuccess) return e;
    int n = 0;
    cfg.gridDim = dim3(C);
    cfg.dynamicSmemBytes = kLinSmemMax;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = smem;
    room[dev][C] = n > 0 ? n : 1;
  }
  const int clusters = units < room[dev][C] ? units : room[dev][C];
  cfg.gridDim = dim3(clusters * C);
  return cudaLaunchKernelEx(&cfg, kernel, w, x, L, C);
}

}  // namespace

cudaError_t launch_linear_stream(LinLaunch L, int cluster, int max_units, cudaStream_t stream) {
  const LinearArgs& a = L.a;
  const bool gated = a.act == GBMOE_EPI_SILU_MUL;
  if (L.bn < 16 || L.bn > kMaxBn || L.bn % 16 || cluster < 1 || cluster > kMaxCluster ||
      cluster > L.k_blocks)
    return cudaErrorInvalidValue;
  const uint32_t stage = kLinWBytes + L.bn * 128;
  const uint32_t per = (L.bn + cluster - 1) / cluster;
  const uint32_t red = cluster > 1 ? cluster * per * kLinWRows * 4 : 0;
  const uint32_t scale = a.fp8 ? kLinScaleSlots * L.bn * 4 * (gated ? 2 : 1) : 0;
  const uint32_t tab = (4u * (3 * a.G + 1) + 15) & ~15u, bars = kBars * 8 + 16;
  const uint32_t rest = red + scale + tab + bars + 1024;
  int stages = (int)((kLinSmemMax - rest) / stage);
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages < 2) return cudaErrorInvalidValue;
  L.stages = stages;
  L.red_off = stages * stage;
  L.scale_off = L.red_off + red;
  L.bar_off = L.scale_off + scale;
  L.tab_off = L.bar_off + bars;
  CUtensorMap w, x;
  if (!lin_maps(a, L.bn, &w, &x)) return cudaErrorInvalidValue;
  const size_t smem = stages * stage + rest;
  if (a.fp8)
    return gated ? launch<true, true>(w, x, L, cluster, max_units, smem, stream)
                 : launch<true, false>(w, x, L, cluster, max_units, smem, stream);
  return gated ? launch<false, true>(w, x, L, cluster, max_units, smem, stream)
               : launch<false, false>(w, x, L, cluster, max_units, smem, stream);
}

}  // namespace gbmoe
