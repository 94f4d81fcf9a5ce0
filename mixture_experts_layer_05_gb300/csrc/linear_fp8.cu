// moe_linear / moe_grouped_linear with e4m3 operands for many rows per group.
//
// Every K block of 128 has its own scales, so its product is formed by itself in TMEM (4 MMAs of K = 32)
// and promoted into fp32 registers, while the next K block's runs into the other of two buffers. Here
// the rows of x are on the MMA's M side: a TMEM lane is a row, whose scale is one register, and the
// weights' scale is the same for 128 columns, so that promoting costs one fma a value. (With the
// weights on M, as the other kernels have them, the rows' scales change from column to column, and
// reading them takes shared memory's time from the operands.)
//
// 8192 rows of 7168 to 4096 columns take 224 to 230 us (2.1 PFLOP/s). Two limits hold it at almost the same height:
// products and promotion, which take turns at TMEM's two buffers of 128 x 256 (212 us without the copies),
// and products and copies (216 without the promotion); products alone take 160, copies alone 172. Pairs of
// CTAs (M = 256), whose operands are two thirds, lift the second only: 242 us as single ones then, and 257
// for 217 with 8192 rows in 16 groups, as short groups waste more of them.
//
// Unit: 128 rows of one group by 256 weight rows (SILU_MUL: 128 gate rows and their up rows).
// Warps: 0 TMA, 1 TMEM and MMA, 2..17 epilogue: the four warps of a TMEM lane quarter take 64 columns
// each, of which every thread keeps the running sums of its row (two with 128 columns each: 278 us for 213
// with 8192 gated rows in 16 groups, the same for the dense call); 18 scales: it writes the products of the
// rows' and the weights' scales of a K block beside the TMEM buffer that they belong to.
#include "linear.cuh"

namespace gbmoe {
namespace {

constexpr int kBM = 128, kBN = 256;
constexpr int kEpiWarps = 16;
constexpr int kCols = 64;                        // accumulator columns of an epilogue thread
constexpr int kThreads = 64 + 32 * kEpiWarps + 32;
constexpr uint32_t kABytes = kBM * 128, kBBytes = kBN * 128, kStageBytes = kABytes + kBBytes;
constexpr uint32_t kTmemCols = 512, kStride = 256;
constexpr int kAhead = 4;                        // K blocks that the scales' loads run ahead
constexpr int kPitch = 33;                       // of the 32 x 32 values that an epilogue warp turns
// the two ways out (below): by rows leaves the ring a stage more
constexpr int stages_of(bool by_rows) { return by_rows ? 4 : 3; }
constexpr uint32_t turn_bytes_of(bool by_rows) { return by_rows ? 0 : kEpiWarps * 32 * kPitch * 4; }

// 8 consecutive bf16 values, 16-byte aligned, as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(u[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// The two ways out of a thread's sums, which are of one row. By rows, 16 bytes at a time, for SILU_MUL where
// the alignment allows it (4096 rows of 512 to 6144: 44 us against 61 turned, 8192 rows in 16 groups: 214
// against 241). Else turned in shared memory, so that a lane has a column and the warp's accesses are 64
// bytes of a row, whatever its alignment (the same plain: 43 us by rows and 35 turned, 8192 rows of 7168
// to 4096: 242 and 226; by rows of odd width, 2 bytes at a time, 1879 rows of 256 to 6854: 106 and 20).

// SILU_MUL: 32 gate and 32 up sums of row t, output columns f0 .. f0 + 32.
__device__ __forceinline__ void store_row(const LinearArgs& a, int g, int t, int f0,
                                          float (&acc)[kCols]) {
  const __nv_bfloat16* bias =
      a.bias ? static_cast<const __nv_bfloat16*>(a.bias) + (long long)g * a.N : nullptr;
  const __nv_bfloat16* res =
      a.residual ? static_cast<const __nv_bfloat16*>(a.residual) + t * a.residual_stride : nullptr;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + t * a.out_stride;
  const float rw = a.row_weight ? __ldg(a.row_weight + t) : 1.f;
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    const int f = f0 + c;
    if (f >= a.cols) break;
    float y[8], b[8];
    if (bias) {
      load8(bias + f, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[c + i] += b[i];
      load8(bias + a.cols + f, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[32 + c + i] += b[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = lin_silu(acc[c + i]) * acc[32 + c + i] * rw;
    if (res) {
      load8(res + f, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += b[i];
    }
    *reinterpret_cast<uint4*>(out + f) =
        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                   pack_bf16x2(y[6], y[7]));
  }
}

// A warp's 32 rows from row t0 on, `rows` of them real: lane l has the row t0 + l, columns f0 .. f0 + 64
// (GATED: 32 gate sums, then their 32 up sums).
template <bool GATED>
__device__ __forceinline__ void store_turned(const LinearArgs& a, int g, int t0, int rows, int f0,
                                             float (&acc)[kCols], float* turn) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* bias =
      a.bias ? static_cast<const __nv_bfloat16*>(a.bias) + (long long)g * a.N : nullptr;
  if (GATED) {
    if (bias) {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const int f = min(f0 + c, a.cols - 1);     // columns past the last are not stored
        acc[c] += __bfloat162float(bias[f]);
        acc[32 + c] += __bfloat162float(bias[a.cols + f]);
      }
    }
#pragma unroll
    for (int c = 0; c < 32; ++c) acc[c] = lin_silu(acc[c]) * acc[32 + c];
  }
#pragma unroll
  for (int half = 0; half < (GATED ? 1 : 2); ++half) {
#pragma unroll
    for (int c = 0; c < 32; ++c) turn[lane * kPitch + c] = acc[32 * half + c];
    __syncwarp();
    const int f = f0 + 32 * half + lane;
    if (f < a.cols) {
      const float b = !GATED && bias ? __bfloat162float(bias[f]) : 0.f;
      const long long rs = a.residual_stride, os = a.out_stride;
      const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(a.residual) + t0 * rs + f;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + t0 * os + f;
#pragma unroll 1
      for (int i0 = 0; i0 < rows; i0 += 8) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = turn[(i0 + i) * kPitch + lane] + b;
        if (!GATED) lin_activate(y, a.act);
        if (a.row_weight) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= __ldg(a.row_weight + t0 + min(i0 + i, rows - 1));
        }
        if (a.residual) {
          __nv_bfloat16 res[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i0 + i < rows) res[i] = *r;
            r += rs;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] += __bfloat162float(res[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i0 + i < rows) *o = __float2bfloat16_rn(y[i]);
          o += os;
        }
      }
    }
    __syncwarp();
  }
}

template <bool GATED, bool BY_ROWS>
__global__ void __launch_bounds__(kThreads, 1)
    linear_fp8_kernel(const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ LinLaunch L) {
  constexpr int kTileCols = GATED ? 128 : 256;     // output columns per unit
  constexpr int kStages = stages_of(BY_ROWS);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const LinearArgs& a = L.a;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);
  // [buffer][row][columns 0 .. 127, 128 .. 255 of the tile]
  float2* scales = reinterpret_cast<float2*>(smem + L.scale_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 2);                  // the products and the scales
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
  const int units = groups.units(L.n_tiles);
  const int KB = L.k_blocks;
  int* const status = a.status;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lin_elect()) {
      int s = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const LinUnit w = groups.unit(L, L.n_tiles, u);
        const int row = w.g * a.N + w.nt * kTileCols;
        const int row1 = row + (GATED ? a.cols : 128);
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_fast(empty_bar(s), ph, abort_flag, status)) {
            ok = false;
            break;
          }
          const uint32_t sa = base + s * kStageBytes;
          mbar_expect_tx(full_bar(s), kStageBytes);
          tma_load_3d(sa, &tm_x, full_bar(s), kb * 128, w.m0, 0);
          tma_load_3d(sa + kABytes, &tm_w, full_bar(s), kb * 128, row, 0);
          tma_load_3d(sa + kABytes + kBBytes / 2, &tm_w, full_bar(s), kb * 128, row1, 0);
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
    if (lin_elect()) {
      constexpr uint32_t idesc = idesc_e4m3(kBM, kBN);
      int s = 0, buf = 0;
      uint32_t ph = 0, tph = 1;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_fast(tempty_bar(buf), tph, abort_flag, status) ||
              !wait_fast(full_bar(s), ph, abort_flag, status)) {
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
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;                  // rows [32 quarter, + 32) of the block
    const int part = (warp - 2) >> 2;              // which columns of the accumulator:
    // SILU_MUL gate [32 part, + 32) and up [128 + 32 part, + 32), else [64 part, + 64)
    const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16) + (GATED ? 32 : 64) * part;
    const int r = quarter * 32 + lane;
    float* turn = reinterpret_cast<float*>(smem + L.red_off) + (warp - 2) * 32 * kPitch;
    int buf = 0;
    uint32_t tph = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
      float acc[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
      for (int kb = 0; kb < KB; ++kb) {
        if (!lin_wait(tfull_bar(buf), tph, abort_flag, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = lanes + buf * kStride;
        const float2 sc = scales[buf * kBM + r];
        const float s0 = GATED || part < 2 ? sc.x : sc.y;
#pragma unroll
        for (int c = 0; c < kCols / 16; ++c) {
          uint32_t v[16];
          tmem_ld16(tb + (GATED && c >= 2 ? 96 + 16 * c : 16 * c), v);
          const float k = GATED && c >= 2 ? sc.y : s0;
          tmem_wait_ld16(v);
#pragma unroll
          for (int q = 0; q < 16; q += 2)
            fma2(acc[16 * c + q], acc[16 * c + q + 1], k, k, __uint_as_float(v[q]),
                 __uint_as_float(v[q + 1]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(buf));
        buf ^= 1;
        if (buf == 0) tph ^= 1u;
      }
      if (!ok) break;
      const LinUnit w = groups.unit(L, L.n_tiles, u);
      const int f0 = w.nt * kTileCols + part * (kTileCols / 4), rows = min(32, w.n - quarter * 32);
      if (BY_ROWS) {
        if (lane < rows) store_row(a, w.g, w.m0 + r, f0, acc);
      } else if (rows > 0) {
        store_turned<GATED>(a, w.g, w.m0 + quarter * 32, rows, f0, acc, turn);
      }
    }
  } else {
    // ------------------------------------------------------------ scales
    const int wblocks = (a.N + 127) >> 7;
    int buf = 0;
    uint32_t tph = 1;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const LinUnit w = groups.unit(L, L.n_tiles, u);
      const int b0 = w.nt * (kTileCols / 128), b1 = GATED ? b0 + (a.cols >> 7) : min(b0 + 1, wblocks - 1);
      const float* w0 = a.w_scale + ((long long)w.g * wblocks + b0) * KB;
      const float* w1 = a.w_scale + ((long long)w.g * wblocks + b1) * KB;
      const float* xs = a.x_scale + w.m0 + lane;
      for (int kb0 = 0; ok && kb0 < KB; kb0 += kAhead) {
        float x[kAhead][4], s0[kAhead], s1[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const bool in = kb0 + i < KB;
          s0[i] = in ? __ldg(w0 + kb0 + i) : 0.f;
          s1[i] = in ? __ldg(w1 + kb0 + i) : 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            x[i][q] = in && lane + 32 * q < w.n ? __ldg(xs + (long long)(kb0 + i) * a.T + 32 * q) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (kb0 + i >= KB) break;
          if (!lin_wait(tempty_bar(buf), tph, abort_flag, status)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            scales[buf * kBM + lane + 32 * q] = make_float2(x[i][q] * s0[i], x[i][q] * s1[i]);
          __syncwarp();
          if (lane == 0) mbar_arrive(tfull_bar(buf));
          buf ^= 1;
          if (buf == 0) tph ^= 1u;
        }
      }
    }
  }

  tc_fence_before();
  lin_leave(1, abort_flag);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool GATED, bool BY_ROWS>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& x, const LinLaunch& L, long long units,
                   size_t smem, cudaStream_t stream) {
  auto kernel = linear_fp8_kernel<GATED, BY_ROWS>;
  static bool ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e == cudaSuccess ? cudaErrorInvalidDevice : e;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmemMax);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  const int grid = units < num_sms() ? (int)units : num_sms();
  kernel<<<grid, kThreads, smem, stream>>>(w, x, L);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_fp8(LinLaunch L, long long max_units, cudaStream_t stream) {
  const LinearArgs& a = L.a;
  if (!a.fp8 || L.bn != kBM) return cudaErrorInvalidValue;
  auto on16 = [](const void* p, long long stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0;
  };
  const bool gated = a.act == GBMOE_EPI_SILU_MUL;
  const bool by_rows = gated && on16(a.out, a.out_stride) && (!a.bias || on16(a.bias, a.cols)) &&
                       (!a.residual || on16(a.residual, a.residual_stride));
  L.stages = stages_of(by_rows);
  L.scale_off = L.stages * (int)kStageBytes;
  L.red_off = L.scale_off + 2 * kBM * (int)sizeof(float2);
  L.bar_off = L.red_off + (int)turn_bytes_of(by_rows);
  L.tab_off = L.bar_off + (2 * L.stages + 4) * 8 + 16;
  CUtensorMap w, x;
  if (!lin_map_rows(a, 128, 0, &w) || !lin_map_x(a, kBM, 0, &x)) return cudaErrorInvalidValue;
  const size_t smem = L.tab_off + 4 * (3 * a.G + 1) + 1024;
  if (by_rows) return launch<true, true>(w, x, L, max_units, smem, stream);
  return gated ? launch<true, false>(w, x, L, max_units, smem, stream)
               : launch<false, false>(w, x, L, max_units, smem, stream);
}

}  // namespace gbmoe
