// The choice between the kernels of moe_linear and moe_grouped_linear, and how a call is cut.
#include "linear.cuh"

namespace gbmoe {

namespace {

bool encode(const LinearArgs& a, CUtensorMap* m, const void* p, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  auto enc = tensor_map_encoder();
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc && enc(m, a.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                    const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `rows` rows of K elements, `stride` elements apart.
bool map_rows(const LinearArgs& a, CUtensorMap* m, const void* p, cuuint64_t rows, cuuint64_t stride,
              int box_rows, int kps) {
  const cuuint64_t es = a.fp8 ? 1 : 2, inner = 128 / es, K = a.K;
  const bool whole = kps > 0;
  const cuuint64_t dims[3] = {whole ? inner : K, rows, whole ? K / inner : 1};
  const cuuint64_t strides[2] = {stride * es, 128};
  const cuuint32_t box[3] = {(cuuint32_t)inner, (cuuint32_t)box_rows, (cuuint32_t)(whole ? kps : 1)};
  return encode(a, m, p, 3, dims, strides, box);
}

}  // namespace

bool lin_map_x(const LinearArgs& a, int rows, int kps, CUtensorMap* x) {
  return map_rows(a, x, a.x, a.T, a.x_stride, rows, kps);
}

bool lin_map_rows(const LinearArgs& a, int rows, int kps, CUtensorMap* w) {
  return map_rows(a, w, a.weight, (cuuint64_t)a.G * a.N, a.K, rows, kps);
}

bool lin_map_tiles(const LinearArgs& a, int rows, int kps, CUtensorMap* w) {
  if (a.act != GBMOE_EPI_SILU_MUL) return lin_map_rows(a, rows, kps, w);
  // (k, row of 16, gate or up of each group, block of 16 features, K block)
  const cuuint64_t es = a.fp8 ? 1 : 2, inner = 128 / es, K = a.K, I = a.N / 2;
  const bool whole = kps > 0;
  const cuuint64_t dims[5] = {whole ? inner : K, 16, 2 * (cuuint64_t)a.G, I / 16, whole ? K / inner : 1};
  const cuuint64_t strides[4] = {K * es, I * K * es, 16 * K * es, 128};
  const cuuint32_t box[5] = {(cuuint32_t)inner, 16, 2, (cuuint32_t)rows / 32, (cuuint32_t)(whole ? kps : 1)};
  return encode(a, w, a.weight, 5, dims, strides, box);
}

namespace {

int ceil_div(long long x, long long y) { return (int)((x + y - 1) / y); }

// How the stream kernel cuts a call: tiles of `rows` weight rows, `cluster` CTAs to a tile.
struct StreamCut {
  int bn, cluster, rows;
  double ns;
};

// Groups count as if all of them had rows. A join of partial sums and the cluster's start take about 3.5 us,
// and some more for the sums' size. cluster 0: the device holds no cluster of some size.
StreamCut cut_stream(const LinearArgs& a, int groups, int mean, int k_blocks) {
  const bool gated = a.act == GBMOE_EPI_SILU_MUL;
  StreamCut best = {0, 0, 0, 1e30};
  // Dense: the rows, cut evenly. Groups: room for the larger ones, in steps of 16 up to 64 (16 of 2048
  // to 7168, mean 16: 73.5 us with 64 against 82.6 with 16; mean 2: 65.9 and 66.3).
  const int bn = a.offsets ? 4 * mean : ceil_div(mean, ceil_div(mean, a.fp8 ? 64 : 128));
  best.bn = (bn + 15) & ~15;
  if (a.offsets && best.bn > 64) best.bn = 64;
  const int n = best.bn, grain = gated ? 32 : 8;             // rows per step of R
  const long long blocks = ceil_div(a.T, n) + (a.offsets ? groups - 1 : 0);
  for (int C = 1; C <= 8 && C <= k_blocks; ++C) {
    const int room = linear_stream_room(a, n, C);
    if (room < 1) return StreamCut{n, 0, 0, 0};
    const int kb = ceil_div(k_blocks, C);
    for (int rounds = 1; rounds <= 8; ++rounds) {
      const long long tiles = (long long)room * rounds / blocks;  // of one group's rows
      int R = tiles < 1 ? 129 : ceil_div(a.N, tiles);
      R = ceil_div(R < 8 ? 8 : R, grain) * grain;
      if (gated && a.fp8 && R == 96) R = 128;      // a tile has one scale block of either kind
      if (R > 128) {
        if (rounds < 8) continue;
        R = 128;
      }
      const long long units = blocks * ceil_div(a.N, R);
      // the weights of a group's further row blocks come from L2
      const long long line = lin_line_ns(units, room, lin_unit_ns(a.fp8, gated, R, n, kb),
                                         (long long)R * a.K * (a.fp8 ? 1 : 2) * groups / blocks);
      const double ns = line + (C > 1 ? ceil_div(units, room) * (3500 + n * R / 20.0) : 0);
      if (ns < best.ns * 0.98) {
        best.ns = ns;
        best.cluster = C;
        best.rows = R;
      }
    }
  }
  return best;
}

// How the kernels for many rows cut it: units of 256 weight rows and `bn` rows of x. A K block of a unit
// takes the e4m3 kernel some 500 ns (128 rows, one CTA; a unit's way out 3 us more), pairs of CTAs the
// MMAs' 1.1 ns a row, or what the issue of its copies takes. Half of the groups count as ending in a block of their own, and
// all as having one.
struct WideCut {
  int bn, tiles;
  double ns;
};

WideCut cut_wide(const LinearArgs& a, int groups, int k_blocks) {
  WideCut best = {0, ceil_div(a.cols, a.act == GBMOE_EPI_SILU_MUL ? 128 : 256), 1e30};
  const double hbm = (double)groups * a.N * a.K * (a.fp8 ? 1 : 2) / 6700;
  const int most = a.fp8 ? 128 : 256;
  for (int cut = 1; cut <= (a.fp8 ? 1 : 4); ++cut) {
    // dense: the rows, cut evenly into up to four times as many blocks as needed
    const int rows = a.offsets || a.fp8 ? most / cut : ceil_div(a.T, (long long)cut * ceil_div(a.T, most));
    const int bn = a.fp8 ? most : (rows + 31) & ~31;
    if (bn < 64 && cut > 1) break;
    const int some = ceil_div(a.T, bn) + (a.offsets ? groups / 2 : 0);
    const long long blocks = some > groups ? some : groups;
    const double block = 9 * bn / 8 > 140 + bn / 8 ? 9 * bn / 8 : 140 + bn / 8;
    const double one = a.fp8 ? 500.0 * k_blocks + 3000 : block * k_blocks;
    const double run = one * ceil_div(blocks * best.tiles, num_sms() / (a.fp8 ? 1 : 2));
    const double ns = run > hbm ? run : hbm;
    if (ns < best.ns) {
      best.ns = ns;
      best.bn = bn;
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
  LinLaunch L = {};
  L.a = a;
  L.k_blocks = (a.K * (a.fp8 ? 1 : 2) + 127) / 128;
  const bool gated = a.act == GBMOE_EPI_SILU_MUL;
  const int mean = ceil_div(a.T, a.G);
  const int groups = a.G < a.T ? a.G : a.T;                  // with rows, at most

  // Few rows or many: by the modelled times. Measured, stream and many (us): K = N = 4096, bf16, 64 rows
  // 12.5 and 14.6, 128 rows 17.6 and 14.8; 96 rows of 2048 to 2048 10.8 and 9.3; e4m3, 128 rows of 4096 to
  // 4096 15.3 and 21.4, 160 to 16384 47.4 and 24.7; 16 groups of 2048 to 7168, mean 32 76.9 and 79.4,
  // mean 64 88.5 and 81.6; e4m3, mean 8 42.6 and 44.1, mean 16 59.7 and 45.5. Where HBM bounds both the few
  // rows' kernel is ahead (4 rows of 4096 to 24576 38.6 and 41.3), and of small groups fewer may have rows
  // than the model counts, which suits it too; above 96 rows its ring gets short, and it has to be
  // well ahead.
  const WideCut wide = cut_wide(a, groups, L.k_blocks);
  bool many = mean > (a.offsets ? 128 : 4096);
  StreamCut cut = {};
  if (!many) {
    cut = cut_stream(a, groups, mean, L.k_blocks);
    if (cut.cluster < 1) return cudaErrorInvalidConfiguration;
    many = cut.ns > (mean <= (a.offsets ? 8 : 64) ? 1.15 : mean <= 96 ? 1.0 : 0.7) * wide.ns;
  }
  if (many) {
    L.n_tiles = wide.tiles;
    L.gm = 16;
    L.bn = wide.bn;
    const long long units = ((long long)ceil_div(a.T, L.bn) + groups - 1) * L.n_tiles;
    return a.fp8 ? launch_linear_fp8(L, units, stream) : launch_linear_pair(L, units, stream);
  }
  L.bn = cut.bn;
  L.gm = 1 << 16;
  L.cluster = cut.cluster;
  L.rows[0] = cut.rows;
  L.choices = 1;
  if (a.offsets) {                                 // the kernel cuts by the groups that it finds
    const int step = a.fp8 && gated ? 64 : 32;     // (such a tile has one scale block of either kind)
    L.choices = 0;
    for (int R = 128; R >= 64; R -= step) L.rows[L.choices++] = R;
    L.rows[L.choices++] = 32;
  }
  const int least = L.rows[L.choices - 1];
  L.n_tiles = ceil_div(a.cols, gated ? least / 2 : least);
  const long long blocks = ceil_div(a.T, L.bn) + (a.offsets ? groups - 1 : 0);
  return launch_linear_stream(L, blocks * L.n_tiles, stream);
}

}  // namespace gbmoe
