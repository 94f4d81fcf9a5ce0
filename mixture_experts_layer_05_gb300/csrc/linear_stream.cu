// moe_linear / moe_grouped_linear for few rows per group: bound by reading the weights.
//
// The weights come at HBM's rate when every SM reads for the same time, and one thread can issue the
// copies fast enough: 48 CTAs drew 6.1 TB/s with stages of 37 KB, but a stage costs the issuing threads
// near 200 ns whatever its size. So the tile is cut to the SMs rather than to the MMA: a unit is R <= 128
// weight rows by at most bn rows of x, where R is such that the units come out in whole rounds, and a
// copy takes several K blocks of them. The MMA (tcgen05.mma, M = 128) runs over R rows and over what
// lies behind them in shared memory, whose TMEM lanes nobody reads. (Plain tiles of up to 64 rows run with
// M = 64: with few columns an MMA takes as long as its weight rows' operands, 23 cycles instead of 39.)
//
// Where the rows of x are many against R, their reading and the MMAs cost more than the weights; there a
// cluster of C CTAs takes a tile of C times the rows and cuts its K blocks into C ranges. The C partial
// sums are joined through distributed shared memory: each CTA sends the columns that CTA d finishes to d
// (one bulk copy each), which adds them in the order of the ranges, so that the result does not depend
// on timing and nothing is kept in a workspace between calls.
//
// Graph replay: 4 rows of 4096 to 6144 columns 11.8 us (HBM 7.4), to 24576 32.7 (29.7), 96 to 4096 14.9 (5.3),
// 24 rows in 16 groups, 10 of them with rows, of 7168 to 4096 gated 94 (86.7); e4m3, 16 rows of
// 7168 to 6144 12.4 (6.5). What is left is the start, 2.5 us to the first weights, and 2.5 us of launch
// and way out.
//
// Warps: 0 TMA, 1 TMEM and MMA, 2..9 epilogue (two per TMEM lane quarter, alternating by 16 columns), 10
// (e4m3) scales. e4m3 products are promoted to fp32 with their scales K block by K block, as the FP8
// layer's are: each K block of a stage has its own TMEM columns.
#include "linear.cuh"

namespace gbmoe {
namespace {

constexpr int kMaxBn = 128, kMaxBnFp8 = 64;      // (e4m3 keeps its sums in registers)
constexpr int kMaxCluster = kLinMaxCluster;
constexpr int kMaxStages = 16;
constexpr int kMaxKps = 8;                       // K blocks per stage
constexpr int kXMaps = 2;                        // x boxes of bn and of 8 rows
constexpr int kWMaps = kLinChoices;              // weight boxes of L.rows[i] rows
constexpr uint32_t kTmemCols = 512;
constexpr int kEpiWarps = 8;
constexpr int kBufsMax = 8;                      // TMEM buffers
constexpr int kScaleSlots = 4;                   // e4m3: stages of scales in flight

constexpr int threads_of(bool fp8) { return 64 + 32 * kEpiWarps + (fp8 ? 32 : 0); }
// barriers: full, empty per stage; tfull, tempty per TMEM buffer; partial sums received, sent ones
// consumed; the epilogue's warps; scales full, empty per slot
constexpr int kBars = 2 * kMaxStages + 2 * kBufsMax + 3 + 2 * kScaleSlots;

struct Maps {
  CUtensorMap w[kWMaps];
  CUtensorMap x[kXMaps];
};

// Shared memory to the shared memory of a CTA of the cluster, counted on a barrier there.
__device__ __forceinline__ void copy_to_cluster(uint32_t dst, uint32_t src, uint32_t bytes,
                                                uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Scales of a slot: for K block j of the stage and row c, the products with the two weight blocks that
// a tile can meet (gate and up; or the blocks before and behind a border of 128 rows), four rows of
// one next to four of the other, so that lanes of both kinds read without conflicts.
__device__ __forceinline__ int scale_at(int bn, int j, int c, int kind) {
  return j * 2 * bn + (c >> 2) * 8 + kind * 4 + (c & 3);
}

// CHUNKS: runs of 16 columns that an epilogue warp holds, for bn up to 32 * CHUNKS.
template <bool FP8, bool GATED, int CHUNKS>
__global__ void __launch_bounds__(threads_of(FP8), 1)
    linear_stream_kernel(const __grid_constant__ Maps maps, const __grid_constant__ LinLaunch L) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const LinearArgs& a = L.a;
  const int C = L.cluster, bn = L.bn, stages = L.stages, kps = L.kps;
  const int w_rows = L.rows[0];                    // the weights' room in a stage, per K block
  const uint32_t stage_bytes = (uint32_t)kps * (w_rows + bn) * 128;
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
  const uint32_t rempty_bar = rfull_bar + 8u, meet_bar = rempty_bar + 8u;
  auto sfull_bar = [&](int s) { return meet_bar + 8u + 8u * s; };
  auto sempty_bar = [&](int s) { return meet_bar + 8u + 8u * (kScaleSlots + s); };
  // TMEM: two accumulators, or a stage's K block products side by side
  uint32_t stride = 16;
  while ((int)stride < bn) stride *= 2;
  const uint32_t buf_cols = FP8 ? stride * kps : stride;
  const int bufs = FP8 ? min(kBufsMax, (int)(kTmemCols / buf_cols)) : 2;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int first = blockIdx.x / C, step = gridDim.x / C;
  const int kb0 = (int)((long long)rank * L.k_blocks / C);
  const int kb1 = (int)((long long)(rank + 1) * L.k_blocks / C);
  const uint64_t policy = l2_evict_first_policy();
  // in registers: behind an asm statement that touches memory, the launch's values are loaded again
  const int out_features = a.N;
  const bool whole = L.whole != 0, grouped = a.offsets != nullptr;
  int* const status = a.status;

  // One stage: the K blocks from kb on of a tile of R weight rows (the choice `pick`).
  auto fill = [&](const LinUnit& w, int R, int pick, int kb, int s) {
    const int nk = min(kps, kb1 - kb);
    const bool few = grouped && w.n <= 8;
    const CUtensorMap* tw = &maps.w[pick];
    const CUtensorMap* tx = &maps.x[few ? 1 : 0];
    const int xr = few ? 8 : bn;
    const uint32_t sw = base + s * stage_bytes, sx = sw + (uint32_t)(kps * w_rows) * 128;
    const uint32_t fb = full_bar(s);
    const int nt = w.nt * (GATED ? R / 32 : R), row = w.g * out_features + nt;
    // a box is always whole: K blocks past the end come as zeros, and those of another CTA's range
    // are read for nothing
    mbar_expect_tx(fb, (uint32_t)((whole ? kps : nk) * (R + xr)) * 128u);
    constexpr int kElems = FP8 ? 128 : 64;
    const int turns = whole ? 1 : nk;
    for (int j = 0; j < turns; ++j) {
      const int x0 = whole ? 0 : (kb + j) * kElems, z = whole ? kb : 0;
      const uint32_t dst = sw + (uint32_t)(j * R) * 128;
      // weights that no other unit reads go first from L2
      if (GATED) {
        if (w.alone) tma_load_5d_hint(dst, tw, fb, x0, 0, 2 * w.g, nt, z, policy);
        else tma_load_5d(dst, tw, fb, x0, 0, 2 * w.g, nt, z);
      } else {
        if (w.alone) tma_load_3d_hint(dst, tw, fb, x0, row, z, policy);
        else tma_load_3d(dst, tw, fb, x0, row, z);
      }
      tma_load_3d(sx + (uint32_t)(j * xr) * 128, tx, fb, x0, w.m0, z);
    }
  };

  int early = 0;                                   // stages filled before the barrier below
  if (warp == 0) {
    // a lane for each: one thread's chain of them is a quarter of a microsecond
    if (lane < stages) {
      mbar_init(full_bar(lane), 1);
      mbar_init(empty_bar(lane), 1);
    }
    if (lane < bufs) {
      mbar_init(tfull_bar(lane), 1);
      mbar_init(tempty_bar(lane), kEpiWarps);
    }
    if (lane < kScaleSlots) {
      mbar_init(sfull_bar(lane), 1);
      mbar_init(sempty_bar(lane), kEpiWarps);
    }
    if (lane == 0) {
      mbar_init(rfull_bar, 1);
      mbar_init(rempty_bar, kEpiWarps * C);
      mbar_init(meet_bar, kEpiWarps);
      *abort_flag = 0;
    }
    fence_mbar_init();
  }
  if (!a.offsets && warp == 0) {
    // one group of known rows: the first loads start now
    const int blocks = (a.T + bn - 1) / bn;
    if (first < blocks * L.n_tiles) {
      early = min(stages, (kb1 - kb0 + kps - 1) / kps);
      __syncwarp();                                // all lanes' barriers are there
      if (lin_elect()) {
        const LinUnit w = LinGroups::place(L, L.n_tiles, first, 0, 0, blocks, 0, a.T);
        for (int i = 0; i < early; ++i) fill(w, w_rows, 0, kb0 + i * kps, i);
      }
      __syncwarp();
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  LinGroups groups(reinterpret_cast<int*>(smem + L.tab_off), a.G);
  groups.load(L);
  tc_fence_before();
  if (C > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  int R = L.rows[0], pick = 0, n_tiles = L.n_tiles;
  if (grouped) {
    // all CTAs have to come to the same tile, so nothing of a CTA's own goes in here
    const int xr = (a.T + a.G - 1) / a.G <= 8 ? 8 : bn;
    pick = lin_pick(L.rows, L.choices, FP8, GATED, a.cols, L.k_blocks, C, xr, groups.before[a.G], step, &n_tiles);
    R = L.rows[pick];
  }
  const int units = groups.units(n_tiles);
  const int tile_cols = GATED ? R / 2 : R;
  const bool half_m = !GATED && R <= 64;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lin_elect()) {
      int s = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int u = first; ok && u < units; u += step) {
        const LinUnit w = groups.unit(L, n_tiles, u);
        for (int kb = kb0; kb < kb1; kb += kps) {
          if (early > 0) {
            --early;                               // on its way already
          } else {
            if (!wait_fast(empty_bar(s), ph, abort_flag, status)) {
              ok = false;
              break;
            }
            fill(w, R, pick, kb, s);
          }
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
    if (lin_elect()) {
      int s = 0, buf = 0;
      uint32_t ph = 0, tph = 1;
      bool ok = true;
      for (int u = first; ok && u < units; u += step) {
        const LinUnit w = groups.unit(L, n_tiles, u);
        const int n = (w.n + 15) & ~15;
        const uint32_t idesc = FP8 ? idesc_e4m3(half_m ? 64 : 128, n) : idesc_bf16(half_m ? 64 : 128, n);
        const uint32_t step_w = (uint32_t)R * 8;   // a K block's weights and rows, in 16-byte units
        const uint32_t step_x = (uint32_t)(grouped && w.n <= 8 ? 8 : bn) * 8;
        for (int kb = kb0; kb < kb1; kb += kps) {
          if (((FP8 || kb == kb0) && !wait_fast(tempty_bar(buf), tph, abort_flag, status)) ||
              !wait_fast(full_bar(s), ph, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sw = base + s * stage_bytes;
          uint64_t dw = sdesc_sw128(sw), dx = sdesc_sw128(sw + (uint32_t)(kps * w_rows) * 128);
          uint32_t d = tmem_base + buf * buf_cols;
          const int nk = min(kps, kb1 - kb);
          uint32_t more = FP8 || kb == kb0 ? 0u : 1u;
          for (int j = 0; j < nk; ++j) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (FP8) mma_e4m3(d, dw + 2 * kk, dx + 2 * kk, idesc, kk != 0 ? 1u : 0u);
              else mma_bf16(d, dw + 2 * kk, dx + 2 * kk, idesc, kk != 0 ? 1u : more);
            }
            more = 1u;
            dw += step_w;
            dx += step_x;
            if (FP8) d += stride;
          }
          mma_commit(empty_bar(s));
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
          if (FP8 || kb + kps >= kb1) {
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
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const int spot = quarter * 32 + lane;
    // the lane's weight row: with M = 64, D's rows are the first 16 lanes of every quarter
    const int row = !half_m ? spot : lane < 16 ? quarter * 16 + lane : kLinWRows;
    // e4m3 with one run of columns: the two warps of a quarter take every other K block instead
    const bool halves = FP8 && bn == 16;
    float* other = reinterpret_cast<float*>(smem + L.half_off);  // [column][128 rows] of the second one
    float* sent = reinterpret_cast<float*>(smem + L.red_off);   // [column][w_rows]
    float* got = sent + bn * w_rows;                            // [rank][column][w_rows]
    const int got_cols = (bn + C - 1) / C;
    int buf = 0, slot = 0;
    uint32_t tph = 0, sph = 0, rph = 0, mph = 0;
    bool ok = true;
    // the epilogue's warps meet, in bounded time as all waits
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet_bar);
      const bool met = lin_wait(meet_bar, mph, abort_flag, status);
      mph ^= 1u;
      return met;
    };
    for (int u = first; ok && u < units; u += step) {
      const LinUnit w = groups.unit(L, n_tiles, u);
      const int f0 = w.nt * tile_cols;             // the tile's first output column
      LinLane l = LinLane::make<GATED>(a, w.g, f0 + quarter * (GATED || half_m ? 16 : 32));
      l.in = l.in && row < R;
      const int per = (w.n + C - 1) / C;           // columns that each CTA finishes
      const int mine = min(per, w.n - rank * per);
      // the first run of columns that this warp finishes; further ones are brought to L2
      constexpr int kStore = GATED ? 8 : 16;
      LinExtra<GATED, kStore> extra;
      extra.fetch(a, l, w.m0 + rank * per + 16 * part, mine - 16 * part);
      if (a.residual && l.in && mine > 32)
        for (int c = 32 + part; c < mine; c += 2)
          lin_prefetch(static_cast<const __nv_bfloat16*>(a.residual) +
                      (long long)(w.m0 + rank * per + c) * a.residual_stride + l.f);
      float acc[FP8 ? CHUNKS * 16 : 16];
      if (FP8) {
        // which of the slot's two products this lane's weight row has
        const int kind = GATED ? lane >> 4 : ((f0 + row) >> 7) - (f0 >> 7);
#pragma unroll
        for (int i = 0; i < CHUNKS * 16; ++i) acc[i] = 0.f;
        for (int kb = kb0; kb < kb1; kb += kps) {
          if (!lin_wait(sfull_bar(slot), sph, abort_flag, status) ||
              !lin_wait(tfull_bar(buf), tph, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int nk = min(kps, kb1 - kb);
          const float* sc = scales + slot * kps * 2 * bn;
          const uint32_t t0 = lanes + buf * buf_cols;
          // two products on their way from TMEM at a time: of two K blocks, or (one per stage) of two
          // runs of columns
          auto load = [&](int j, int col, uint32_t (&v)[16]) { tmem_ld16(t0 + j * stride + col, v); };
          auto add = [&](float* y, int j, int col, uint32_t (&v)[16]) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 k =
                  *reinterpret_cast<const float4*>(sc + scale_at(bn, j, col + 4 * q, kind & 1));
              fma2(y[4 * q], y[4 * q + 1], k.x, k.y, __uint_as_float(v[4 * q]),
                   __uint_as_float(v[4 * q + 1]));
              fma2(y[4 * q + 2], y[4 * q + 3], k.z, k.w, __uint_as_float(v[4 * q + 2]),
                   __uint_as_float(v[4 * q + 3]));
            }
          };
          uint32_t v0[16], v1[16];
          if (halves) {
            for (int j = (kb - kb0 + part) & 1; j < nk; j += 4) {
              load(j, 0, v0);
              if (j + 2 < nk) load(j + 2, 0, v1);
              tmem_wait_ld16(v0);
              add(acc, j, 0, v0);
              if (j + 2 < nk) {
                tmem_wait_ld16(v1);
                add(acc, j + 2, 0, v1);
              }
            }
          } else if (nk == 1) {
#pragma unroll
            for (int c = 0; c < CHUNKS; c += 2) {
              const int col = 16 * (2 * c + part);
              if (col >= w.n) break;
              const bool two = CHUNKS > 1 && col + 32 < w.n;
              load(0, col, v0);
              if (two) load(0, col + 32, v1);
              tmem_wait_ld16(v0);
              add(acc + (FP8 ? 16 * c : 0), 0, col, v0);
              if (two) {
                tmem_wait_ld16(v1);
                add(acc + (FP8 && CHUNKS > 1 ? 16 * c + 16 : 0), 0, col + 32, v1);
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
              const int col = 16 * (2 * c + part);
              if (col >= w.n) break;
              for (int j = 0; j < nk; j += 2) {
                load(j, col, v0);
                if (j + 1 < nk) load(j + 1, col, v1);
                tmem_wait_ld16(v0);
                add(acc + (FP8 ? 16 * c : 0), j, col, v0);
                if (j + 1 < nk) {
                  tmem_wait_ld16(v1);
                  add(acc + (FP8 ? 16 * c : 0), j + 1, col, v1);
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(tempty_bar(buf));
            mbar_arrive(sempty_bar(slot));
          }
          if (++buf == bufs) {
            buf = 0;
            tph ^= 1u;
          }
          if (++slot == kScaleSlots) {
            slot = 0;
            sph ^= 1u;
          }
        }
      } else if (!lin_wait(tfull_bar(buf), tph, abort_flag, status)) {
        ok = false;
      }
      if (!ok) break;
      tc_fence_after();
      if (halves) {
        if (part == 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) other[i * kLinWRows + spot] = acc[i];
        }
        if (!meet()) {
          ok = false;
          break;
        }
        if (part == 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[i] += other[i * kLinWRows + spot];
        }
        if (u + step < units && !meet()) {         // before the next unit's are written
          ok = false;
          break;
        }
      }
      // what the unit before sent has been added up, here and by the others
      if (C > 1 && u != first && !lin_wait<true>(rempty_bar, rph ^ 1u, abort_flag, status)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int col = 16 * (2 * c + part);
        if (col >= w.n) break;
        float v[16];
        if (FP8) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = acc[FP8 ? 16 * c + i : 0];
        } else {
          uint32_t t[16];
          tmem_ld16(lanes + buf * buf_cols + col, t);
          tmem_wait_ld16(t);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(t[i]);
        }
        if (C == 1) {
          if (c > 0) extra.fetch(a, l, w.m0 + col, w.n - col);
          lin_store<GATED, kStore>(a, l, w.m0 + col, w.n - col, v, extra);
        } else if (row < w_rows) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (col + i < w.n) sent[(col + i) * w_rows + row] = v[i];
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
        fence_async_shared();
        if (!meet()) {
          ok = false;
          break;
        }
        if (warp == 2 && lane < C) {
          // the others' sums of this CTA's columns, and this one's of theirs
          const uint32_t col_bytes = w_rows * 4;
          if (lane == rank) {
            mbar_expect_tx(rfull_bar, max(mine, 0) * (C - 1) * col_bytes);
          } else {
            const int theirs = min(per, w.n - lane * per);
            if (theirs > 0)
              copy_to_cluster(mapa_shared(smem_addr(got + rank * got_cols * w_rows), lane),
                              smem_addr(sent + lane * per * w_rows), theirs * col_bytes,
                              mapa_shared(rfull_bar, lane));
          }
        }
        if (!lin_wait<true>(rfull_bar, rph, abort_flag, status)) {
          ok = false;
          break;
        }
        for (int c0 = part * 16; c0 < mine; c0 += 32) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
          if (row < w_rows) {
            for (int s = 0; s < C; ++s) {
              const float* from = s == rank ? sent + rank * per * w_rows : got + s * got_cols * w_rows;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (c0 + i < mine) v[i] += from[(c0 + i) * w_rows + row];
            }
          }
          if (c0 >= 32) extra.fetch(a, l, w.m0 + rank * per + c0, mine - c0);
          lin_store<GATED, kStore>(a, l, w.m0 + rank * per + c0, mine - c0, v, extra);
        }
        if (u + step < units) {
          __syncwarp();
          if (lane < C) mbar_arrive_cluster(mapa_shared(rempty_bar, lane));
        }
        rph ^= 1u;
      }
    }
  } else if (FP8) {
    // ------------------------------------------------------------ scales
    const int wblocks = (a.N + 127) >> 7;
    // A stage's scales, fetched while the stage before is on its way: the loads' latency, paid between a
    // free slot and the next, would be longer than a stage takes (128 rows in 16 groups, 2048 to 7168:
    // 38 us).
    float v[kMaxKps][CHUNKS], s0[kMaxKps], s1[kMaxKps];
    auto fetch = [&](const LinUnit& w, int kb) {
      const int b0 = (w.nt * tile_cols) >> 7;
      const int b1 = GATED ? b0 + (a.cols >> 7) : min(b0 + 1, wblocks - 1);
      const float* w0 = a.w_scale + ((long long)w.g * wblocks + b0) * L.k_blocks + kb;
      const float* w1 = a.w_scale + ((long long)w.g * wblocks + b1) * L.k_blocks + kb;
      const float* xs = a.x_scale + (long long)kb * a.T + w.m0 + lane;
#pragma unroll
      for (int j = 0; j < kMaxKps; ++j) {
        const bool in = j < kps && kb + j < kb1;
        s0[j] = in ? __ldg(w0 + j) : 0.f;
        s1[j] = in ? __ldg(w1 + j) : 0.f;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
          v[j][i] = in && lane + 32 * i < w.n ? __ldg(xs + (long long)j * a.T + 32 * i) : 0.f;
      }
    };
    int slot = 0;
    uint32_t ph = 1;
    bool ok = true;
    LinUnit w;
    if (first < units) {
      w = groups.unit(L, n_tiles, first);
      fetch(w, kb0);
    }
    for (int u = first; ok && u < units; u += step) {
      for (int kb = kb0; kb < kb1; kb += kps) {
        if (!lin_wait(sempty_bar(slot), ph, abort_flag, status)) {
          ok = false;
          break;
        }
        float* dst = scales + slot * kps * 2 * bn;
#pragma unroll
        for (int j = 0; j < kMaxKps; ++j) {
          if (j >= kps) break;
#pragma unroll
          for (int i = 0; i < CHUNKS; ++i) {
            const int c = lane + 32 * i;
            if (c < bn) {
              dst[scale_at(bn, j, c, 0)] = v[j][i] * s0[j];
              dst[scale_at(bn, j, c, 1)] = v[j][i] * s1[j];
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull_bar(slot));
        if (kb + kps < kb1) {
          fetch(w, kb + kps);
        } else if (u + step < units) {
          w = groups.unit(L, n_tiles, u + step);
          fetch(w, kb0);
        }
        if (++slot == kScaleSlots) {
          slot = 0;
          ph ^= 1u;
        }
      }
    }
  }

  tc_fence_before();
  lin_leave(C, abort_flag);     // no CTA leaves while another may still write to it or read it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

cudaLaunchConfig_t config(bool fp8, int C, unsigned grid, size_t smem, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads_of(fp8));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  if (C > 1) {
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = C;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cfg;
}

// Prepares the kernel on the current device and finds its clusters there, once.
template <bool FP8, bool GATED, int CHUNKS>
int room(int C) {
  static int cached[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (!cached[dev][C]) {
    auto kernel = linear_stream_kernel<FP8, GATED, CHUNKS>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmemMax) !=
        cudaSuccess)
      return 0;
    int n = num_sms();
    if (C > 1) {
      cudaLaunchAttribute attr;
      const cudaLaunchConfig_t cfg = config(FP8, C, C, kLinSmemMax, nullptr, &attr);
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
    }
    cached[dev][C] = n > 0 ? n : 1;
  }
  return cached[dev][C];
}

template <bool FP8, bool GATED, int CHUNKS>
cudaError_t launch(const Maps& maps, const LinLaunch& L, unsigned grid, size_t smem,
                   cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(FP8, L.cluster, grid, smem, stream, &attr);
  return cudaLaunchKernelEx(&cfg, linear_stream_kernel<FP8, GATED, CHUNKS>, maps, L);
}

}  // namespace

int linear_stream_room(const LinearArgs& a, int bn, int size) {
  if (size < 1 || size > kMaxCluster) return 0;
  const bool gated = a.act == GBMOE_EPI_SILU_MUL;
  if (a.fp8 && bn <= 32) return gated ? room<true, true, 1>(size) : room<true, false, 1>(size);
  if (a.fp8) return gated ? room<true, true, 2>(size) : room<true, false, 2>(size);
  return gated ? room<false, true, 4>(size) : room<false, false, 4>(size);
}

cudaError_t launch_linear_stream(LinLaunch L, long long max_units, cudaStream_t stream) {
  const LinearArgs& a = L.a;
  const bool gated = a.act == GBMOE_EPI_SILU_MUL;
  const int C = L.cluster, most_rows = L.rows[0];
  if (L.bn < 16 || L.bn > (a.fp8 ? kMaxBnFp8 : kMaxBn) || L.bn % 16 || C < 1 || C > kMaxCluster || C > L.k_blocks ||
      L.choices < 1 || L.choices > kWMaps)
    return cudaErrorInvalidValue;
  for (int i = 0; i < L.choices; ++i) {
    const int r = L.rows[i];
    // tiles start on the swizzle's 8 rows; gated ones are whole blocks of 16 features, and have one
    // scale block of either kind
    if (r < 8 || r > most_rows || r > kLinWRows || r % 8 || (gated && r % 32) ||
        (gated && a.fp8 && 128 % (r / 2)))
      return cudaErrorInvalidValue;
  }
  const uint32_t w_rows = most_rows, per_k = (w_rows + L.bn) * 128;
  const uint32_t red = C > 1 ? (L.bn + C * ((L.bn + C - 1) / C)) * w_rows * 4 : 0;
  const uint32_t tab = (4u * (3 * a.G + 1) + 15) & ~15u, bars = kBars * 8 + 16;
  // A stage's round trip, barriers, copies and commit, takes one thread or the other near 200 ns, some
  // 25 KB of HBM's time: large stages, of which three still fit
  const uint32_t range = (L.k_blocks + C - 1) / C;
  const uint32_t free_bytes = kLinSmemMax - 1024 - (red + tab + bars > kLinWBytes ? red + tab + bars : kLinWBytes);
  uint32_t kps = free_bytes / 3 / per_k;
  if (kps > range) kps = range;
  if (kps > (uint32_t)kMaxKps) kps = kMaxKps;
  if (a.fp8)
    while (kps > 1 && kps * L.bn > 128) --kps;
  if (kps < 1) kps = 1;
  const uint32_t stage = kps * per_k;
  const uint32_t scale = a.fp8 ? kScaleSlots * kps * 2 * L.bn * 4 : 0;
  const uint32_t half = a.fp8 && L.bn == 16 ? 16 * kLinWRows * 4 : 0;
  // the MMA reads 128 rows from each K block's weights on: behind the last of them too
  const uint32_t over = kLinWBytes, rest = red + scale + half + tab + bars;
  const uint32_t behind = rest > over ? rest : over;
  if (kLinSmemMax < 1024 + behind + 2 * stage) return cudaErrorInvalidValue;
  uint32_t stages = (kLinSmemMax - 1024 - behind) / stage;
  if (stages > (uint32_t)kMaxStages) stages = kMaxStages;
  L.whole = lin_whole(a);
  L.kps = (int)kps;
  L.stages = (int)stages;
  L.red_off = (int)(stages * stage);
  L.scale_off = L.red_off + (int)red;
  L.half_off = L.scale_off + (int)scale;
  L.bar_off = L.half_off + (int)half;
  L.tab_off = L.bar_off + (int)bars;
  Maps maps;
  const int boxed = L.whole ? (int)kps : 0;
  bool ok = lin_map_x(a, L.bn, boxed, &maps.x[0]) &&
            (!a.offsets || lin_map_x(a, 8, boxed, &maps.x[1]));
  for (int i = 0; i < L.choices; ++i) ok = ok && lin_map_tiles(a, L.rows[i], boxed, &maps.w[i]);
  if (!ok) return cudaErrorInvalidValue;
  const int most = linear_stream_room(a, L.bn, C);
  if (most < 1) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)(max_units < most ? max_units : most) * C;
  const size_t smem = 1024 + stages * stage + behind;
  if (a.fp8 && L.bn <= 32)
    return gated ? launch<true, true, 1>(maps, L, grid, smem, stream)
                 : launch<true, false, 1>(maps, L, grid, smem, stream);
  if (a.fp8)
    return gated ? launch<true, true, 2>(maps, L, grid, smem, stream)
                 : launch<true, false, 2>(maps, L, grid, smem, stream);
  return gated ? launch<false, true, 4>(maps, L, grid, smem, stream)
               : launch<false, false, 4>(maps, L, grid, smem, stream);
}

}  // namespace gbmoe
