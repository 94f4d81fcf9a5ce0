// How the dense and grouped products are cut and which kernel runs them, by modelled times. Free of CUDA so
// that it also compiles for the host.
#pragma once

#include "paged_checks.h"

namespace gbmoe {

constexpr int kLinMaxCluster = 8;                // CTAs that cut a unit's K blocks
constexpr int kLinChoices = 4;                   // tiles of weight rows that a grouped call picks from

// A call: T rows of K, G groups of N weight rows. grouped: the device alone knows the rows of each group.
struct LinSize {
  int T, G, K, N;
  bool grouped, gated, fp8;
  int cols() const { return gated ? N / 2 : N; }
};

// The stream kernel's time for a unit of R weight rows and n rows of x over so many K blocks, in ns, fitted
// to measurements at K = N = 4096: a CTA takes 128 bytes a ns from L2 and HBM together; a K block's
// MMAs, whose time goes by their 128 (plain tiles of up to 64: 64) weight rows, and the operands of its
// columns take 90 and 1 (55 and 1.2) a row of x (e4m3: its promotion 50 and 5); a unit's beginning and end
// 300, with e4m3, whose sums leave the registers between two units, 2000.
GBMOE_HD long long lin_unit_ns(bool fp8, bool gated, int R, int n, int k_blocks) {
  const int math = fp8 ? 50 + 5 * n : R <= 64 && !gated ? 55 + 6 * n / 5 : 90 + n;
  return (long long)k_blocks * (R + n > math ? R + n : math) + (fp8 ? 2000 : 300);
}

// The time for `units` of them, `bytes` of weights each, by `step` CTAs or clusters at once: full rounds, in
// which HBM's 6.7 TB/s may be what holds, and a last one, in which each unit takes its own time at least.
GBMOE_HD long long lin_line_ns(long long units, int step, long long unit_ns, long long bytes) {
  const long long all = step * bytes / 6700, full = units / step, rest = units % step;
  const long long last = rest * bytes / 6700;
  return full * (all > unit_ns ? all : unit_ns) + (rest == 0 ? 0 : last > unit_ns ? last : unit_ns);
}

inline int lin_ceil_div(long long x, long long y) { return (int)((x + y - 1) / y); }

// How the stream kernel cuts a call: tiles of `rows` weight rows, `cluster` CTAs to a tile.
struct StreamCut {
  int bn, cluster, rows;
  double ns;
};

// Groups count as if all of them had rows. A join of partial sums and the cluster's start take about 3.5 us,
// and some more for the sums' size. cluster 0: the device holds no cluster of some size.
template <class Room>
StreamCut cut_stream(const LinSize& a, int groups, int mean, int k_blocks, Room room_of) {
  const bool gated = a.gated;
  StreamCut best = {0, 0, 0, 1e30};
  // Dense: the rows, cut evenly. Groups: room for the larger ones, in steps of 16 up to 64 (16 of 2048
  // to 7168, mean 16: 73.5 us with 64 against 82.6 with 16; mean 2: 65.9 and 66.3).
  const int bn = a.grouped ? 4 * mean : lin_ceil_div(mean, lin_ceil_div(mean, a.fp8 ? 64 : 128));
  best.bn = (bn + 15) & ~15;
  if (a.grouped && best.bn > 64) best.bn = 64;
  const int n = best.bn, grain = gated ? 32 : 8;             // rows per step of R
  const long long blocks = lin_ceil_div(a.T, n) + (a.grouped ? groups - 1 : 0);
  for (int C = 1; C <= kLinMaxCluster && C <= k_blocks; ++C) {
    const int room = room_of(n, C);
    if (room < 1) return StreamCut{n, 0, 0, 0};
    const int kb = lin_ceil_div(k_blocks, C);
    for (int rounds = 1; rounds <= 8; ++rounds) {
      const long long tiles = (long long)room * rounds / blocks;  // of one group's rows
      int R = tiles < 1 ? 129 : lin_ceil_div(a.N, tiles);
      R = lin_ceil_div(R < 8 ? 8 : R, grain) * grain;
      if (gated && a.fp8 && R == 96) R = 128;      // a tile has one scale block of either kind
      if (R > 128) {
        if (rounds < 8) continue;
        R = 128;
      }
      const long long units = blocks * lin_ceil_div(a.N, R);
      // the weights of a group's further row blocks come from L2
      const long long line = lin_line_ns(units, room, lin_unit_ns(a.fp8, gated, R, n, kb),
                                         (long long)R * a.K * (a.fp8 ? 1 : 2) * groups / blocks);
      const double ns = line + (C > 1 ? lin_ceil_div(units, room) * (3500 + n * R / 20.0) : 0);
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
// MMAs' 1.1 ns a row, or what the issue of its copies takes. Half of the groups count as ending in a block
// of their own, and all as having one.
struct WideCut {
  int bn, tiles;
  double ns;
};

inline WideCut cut_wide(const LinSize& a, int groups, int k_blocks, int sms) {
  WideCut best = {0, lin_ceil_div(a.cols(), a.gated ? 128 : 256), 1e30};
  const double hbm = (double)groups * a.N * a.K * (a.fp8 ? 1 : 2) / 6700;
  const int most = a.fp8 ? 128 : 256;
  for (int cut = 1; cut <= (a.fp8 ? 1 : 4); ++cut) {
    // dense: the rows, cut evenly into up to four times as many blocks as needed
    const int rows = a.grouped || a.fp8 ? most / cut
                                        : lin_ceil_div(a.T, (long long)cut * lin_ceil_div(a.T, most));
    const int bn = a.fp8 ? most : (rows + 31) & ~31;
    if (bn < 64 && cut > 1) break;
    const int some = lin_ceil_div(a.T, bn) + (a.grouped ? groups / 2 : 0);
    const long long blocks = some > groups ? some : groups;
    const double block = 9 * bn / 8 > 140 + bn / 8 ? 9 * bn / 8 : 140 + bn / 8;
    const double one = a.fp8 ? 500.0 * k_blocks + 3000 : block * k_blocks;
    const double run = one * lin_ceil_div(blocks * best.tiles, sms / (a.fp8 ? 1 : 2));
    const double ns = run > hbm ? run : hbm;
    if (ns < best.ns) {
      best.ns = ns;
      best.bn = bn;
    }
  }
  return best;
}

// A call's kernel and cut. Few rows: linear_stream.cu; many: linear_pair.cu or (e4m3) linear_fp8.cu.
struct LinPlan {
  bool ok;               // false: the device holds no cluster of some size
  bool many;
  int bn;                // rows of x per block
  int n_tiles;           // feature tiles of a group's weights (few: of the smallest choice)
  int cluster;           // few: CTAs that cut K
  int rows[kLinChoices], choices;   // few: weight rows per tile, largest first; the kernel picks, by its groups
  long long units;       // at most
};

// room_of(bn, C): clusters of C CTAs of the few-row kernel that the device holds at once.
template <class Room>
LinPlan lin_plan(const LinSize& a, int sms, Room room_of) {
  LinPlan p = {};
  p.ok = true;
  const int k_blocks = (a.K * (a.fp8 ? 1 : 2) + 127) / 128;
  const int mean = lin_ceil_div(a.T, a.G);
  const int groups = a.G < a.T ? a.G : a.T;                  // with rows, at most

  // Few rows or many: by the modelled times. Measured in one run, graph replay, few and many (us): bf16, 4 rows
  // of 4096 to 24576 32.3 and 36.9; K = N = 4096, 64 rows 12.7 and 14.8, 96 with residual 14.9 and 15.3, 128
  // 17.9 and 15.2; 96 rows of 2048 to 2048 10.7 and 9.6, 64 of 4096 to 16384 24.5 and 25.3; 16 groups of 2048
  // to 7168, mean 4 68.9 and 68.5, 16 73.5 and 73.1, 32 76.7 and 74.3, 64 99.1 and 76.4. e4m3, K = N = 4096,
  // 128 rows 14.7 and 20.1, 160 to 256 17.5 and 20.2 (the rule takes the slower one there); 160 to 16384
  // 44.6 and 24.5; the groups' mean 4 39.6 and 40.3, 8 41.0 and 42.1, 16 42.6 and 43.9 (again), 32 48.6 and 46.4.
  // Where HBM bounds both by the model the few rows' kernel is ahead by up to 14 %, and of small groups fewer
  // may have rows than the model counts, which suits it too: the first factor. Above 96 rows its ring gets
  // short, and it has to be well ahead: the last.
  const WideCut wide = cut_wide(a, groups, k_blocks, sms);
  p.many = mean > (a.grouped ? 128 : 4096);
  StreamCut cut = {};
  if (!p.many) {
    cut = cut_stream(a, groups, mean, k_blocks, room_of);
    p.ok = cut.cluster > 0;
    p.many = cut.ns > (mean <= (a.grouped ? 8 : 64) ? 1.15 : mean <= 96 ? 1.0 : 0.7) * wide.ns;
  }
  if (p.many) {
    p.n_tiles = wide.tiles;
    p.bn = wide.bn;
    p.units = ((long long)lin_ceil_div(a.T, p.bn) + groups - 1) * p.n_tiles;
    return p;
  }
  p.bn = cut.bn;
  p.cluster = cut.cluster;
  p.rows[0] = cut.rows;
  p.choices = 1;
  if (a.grouped) {                                 // the kernel cuts by the groups that it finds
    const int step = a.fp8 && a.gated ? 64 : 32;   // (such a tile has one scale block of either kind)
    p.choices = 0;
    for (int R = 128; R >= 64; R -= step) p.rows[p.choices++] = R;
    p.rows[p.choices++] = 32;
  }
  const int least = p.rows[p.choices - 1];
  p.n_tiles = lin_ceil_div(a.cols(), a.gated ? least / 2 : least);
  const long long blocks = lin_ceil_div(a.T, p.bn) + (a.grouped ? groups - 1 : 0);
  p.units = blocks * p.n_tiles;
  return p;
}

// The tile of a grouped call of few rows with so many row blocks: of the choices, the one whose line of units
// takes least (16 groups of which 10 have rows, 7168 to 4096 gated: 320 tiles of 128 rows took 103 us on 152
// SMs, 430 of 96 95). step: CTAs or clusters; xr: rows of x that a unit reads.
GBMOE_HD int lin_pick(const int* rows, int choices, bool fp8, bool gated, int cols, int k_blocks, int C,
                      int xr, int blocks, int step, int* n_tiles) {
  long long best = 0;
  int pick = 0;
  // A smaller tile is not read faster: the ring holds as many K blocks of it, and fewer bytes.
  const long long unit_ns = lin_unit_ns(fp8, gated, rows[0], xr, (k_blocks + C - 1) / C);
  for (int i = 0; i < choices; ++i) {
    const int r = rows[i], tile = gated ? r / 2 : r;
    const int nt = (cols + tile - 1) / tile;
    const long long u = (long long)blocks * nt;
    if (i > 0 && u > 1 << 30) break;               // units are counted in 32 bits
    const long long cost = lin_line_ns(u, step, unit_ns, (long long)r * k_blocks * 128);
    if (i == 0 || cost < best) {
      best = cost;
      pick = i;
      *n_tiles = nt;
    }
  }
  return pick;
}

}  // namespace gbmoe
