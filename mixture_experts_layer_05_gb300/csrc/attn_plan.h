// How paged attention is cut into work, free of CUDA so that it also compiles for the host.
//
// The rows of one (sequence, kv head) are its new tokens times the G query heads that share
// the head, row = token * G + head; a unit is a block of BR of them, which walks the tiles of
// TK keys that any of its tokens attends (at least one tile, so that rows without keys get
// their zeros). The tiles of all units, in (sequence, kv head, row block) order, form one line
// that is cut into equal ranges, one per CTA: however ragged the lengths are, every CTA reads
// the same number of tiles. A unit that a cut crosses is computed in pieces, each leaving its
// running maximum, sum and unnormalised output in the workspace, joined in order afterwards.
#pragma once

#include "paged_checks.h"

namespace gbmoe {

constexpr int kAttnTK = 128;  // keys per tile

struct AttnShape {
  int G, hkv;      // query heads per kv head, kv heads
  uint32_t g_mul;  // r / G for 0 <= r < 2^31 is the high word of r * g_mul, shifted (G > 1)
  int g_shift;
  int br_shift;    // rows per unit: 1 << br_shift
  int extra;       // cost of a unit beyond its tiles
  // cost of a tile, in units of up to half the rows and in the others
  static constexpr int half = 1, full = 1;
  bool causal;
  int window;
};

// The same with other costs. Functions of the plan take either (a cost of 1 known at compile time
// spares a division where pieces begin).
template <int HALF, int FULL>
struct AttnShapeOf : AttnShape {
  static constexpr int half = HALF, full = FULL;
};

// g_mul = ceil(2^(31 + s) / G), s = ceil(log2 G): division by an invariant integer (Granlund and
// Montgomery); a division instruction sequence per use was a good part of a small call.
inline void set_group(AttnShape& a, int G) {
  int s = 0;
  while ((1 << s) < G) ++s;
  a.G = G;
  a.g_mul = G > 1 ? (uint32_t)(((1ull << (31 + s)) + G - 1) / G) : 0;
  a.g_shift = s - 1;
}
GBMOE_HD int div_group(const AttnShape& a, int r) {
  if (a.G == 1) return r;
#ifdef __CUDA_ARCH__
  return (int)(__umulhi((uint32_t)r, a.g_mul) >> a.g_shift);
#else
  return (int)(((uint64_t)(uint32_t)r * a.g_mul >> 32) >> a.g_shift);
#endif
}

struct UnitKeys {
  int i0, i1;      // first and last token of the unit
  int lo, hi;      // keys that any of them attends: [lo, hi), hi <= lo when none
  int t0, tiles;   // tiles t0 .. t0 + tiles - 1, tile t holding the keys from t * kAttnTK
  int cost;        // of a tile, on the line
};

GBMOE_HD int unit_blocks(const AttnShape& a, int n) {
  return (n * a.G + (1 << a.br_shift) - 1) >> a.br_shift;
}

template <class Shape>
GBMOE_HD UnitKeys unit_keys(const Shape& a, const SeqInfo& q, int rb) {
  UnitKeys u;
  const int r0 = rb << a.br_shift;
  int r1 = r0 + (1 << a.br_shift);
  if (r1 > q.n * a.G) r1 = q.n * a.G;
  u.cost = 2 * (r1 - r0) > 1 << a.br_shift ? a.full : a.half;
  u.i0 = div_group(a, r0);
  u.i1 = div_group(a, r1 - 1);
  u.lo = key_range(q, u.i0, a.causal, a.window).lo;
  u.hi = key_range(q, u.i1, a.causal, a.window).hi;
  if (u.hi <= u.lo) {
    u.hi = u.lo = 0;
    u.t0 = 0;
    u.tiles = 1;
  } else {
    u.t0 = u.lo / kAttnTK;
    u.tiles = (u.hi + kAttnTK - 1) / kAttnTK - u.t0;
  }
  return u;
}

// Length on the line of a unit, and of one kv head of a sequence.
template <class Shape>
GBMOE_HD int unit_length(const Shape& a, const SeqInfo& q, int rb) {
  const UnitKeys u = unit_keys(a, q, rb);
  return u.tiles * u.cost + a.extra;
}
template <class Shape>
GBMOE_HD int seq_length(const Shape& a, const SeqInfo& q) {
  const int blocks = unit_blocks(a, q.n);
  int t = 0;
  GBMOE_ROLLED
  for (int rb = 0; rb < blocks; ++rb) t += unit_length(a, q, rb);
  return t;
}

// The first tile that does not lie before the place `off` of a unit: a cut there ends one piece
// before it and begins the next with it.
template <class Shape>
GBMOE_HD int tile_at(const Shape& a, const UnitKeys& u, int off) {
  if (off <= a.extra) return 0;
  return u.cost == 1 ? off - a.extra : (off - a.extra + u.cost - 1) / u.cost;
}

// CTAs that share a line of length W, about a tile's cost each at least. Where a tile costs 1, a
// range holds a tile, but for ranges within a unit's extra cost, which lies before its tiles: the
// pieces of a unit are in neighbouring CTAs, one each, as attn_decode.cu counts them. With other
// costs a range may also fall within a tile and hold nothing, so that a unit's pieces skip a CTA:
// attn_join_kernel passes over those.
template <class Shape>
GBMOE_HD int line_ctas(const Shape& a, int W, int most) {
  const int n = (W + a.full - 1) / a.full;
  return n < most ? n : most;
}

// A place on the line of tiles.
struct AttnCursor {
  int s, head, rb, off;    // sequence, kv head, row block, length of the unit that is behind
  int left;                // length of this CTA's range that lies ahead
};

// Moves the cursor `rem` further, over row blocks of the sequence q.
template <class Shape>
GBMOE_HD void walk_blocks(const Shape& a, const SeqInfo& q, int rem, AttnCursor& c) {
  GBMOE_ROLLED
  for (;;) {
    const int t = unit_length(a, q, c.rb);
    if (rem < t) break;
    rem -= t;
    ++c.rb;
  }
  c.off = rem;
}

// The part of a unit that one CTA computes.
struct AttnPiece {
  int s, head, rb;
  SeqInfo q;
  UnitKeys u;
  int ta, tb;              // tiles [ta, tb) of the unit, counted from u.t0
  GBMOE_HD bool first() const { return ta == 0; }
  GBMOE_HD bool last() const { return tb == u.tiles; }
  GBMOE_HD bool whole() const { return first() && last(); }
};

// The piece of the sequence q = sequence c.s at the cursor, which moves past it (c.s may then
// be a sequence without rows: the caller skips those). ta == tb: the range ends in the unit's
// extra cost and holds none of its tiles.
template <class Shape>
GBMOE_HD AttnPiece take_piece(const Shape& a, const SeqInfo& q, AttnCursor& c) {
  AttnPiece p;
  p.s = c.s;
  p.head = c.head;
  p.rb = c.rb;
  p.q = q;
  p.u = unit_keys(a, q, c.rb);
  const int len = p.u.tiles * p.u.cost + a.extra;
  const int end = len - c.off > c.left ? c.off + c.left : len;
  p.ta = tile_at(a, p.u, c.off);
  p.tb = tile_at(a, p.u, end);
  c.left -= end - c.off;
  c.off = end;
  if (end == len) {
    c.off = 0;
    if (++c.rb == unit_blocks(a, q.n)) {
      c.rb = 0;
      if (++c.head == a.hkv) {
        c.head = 0;
        ++c.s;
      }
    }
  }
  return p;
}

// CTA c of g takes the range [range_at(c), range_at(c + 1)) of a line of length W.
GBMOE_HD int range_at(int W, int c, int g) { return W / g * c + W % g * c / g; }

// The costs of the launches, whose units have 1 << br_shift rows: 8 or 16 (attn_decode.cu, a tile
// costs 1) or 256 (attn_tc.cu).
//
// Heads of 64 on the tensor cores, a tile of a unit of one half and of two: a chunk of 400 tokens
// among 18 single ones of 3500 keys takes 81, 75, 77, 87 us at 1:1, 4:5, 2:3, 1:2 (bf16), two
// chunks 102, 100, 104, 118. Heads of 128: two chunks 123 us at 1:1, 130 at 4:5.
template <int D>
using AttnTcShape = AttnShapeOf<D == 64 ? 4 : 1, D == 64 ? 5 : 1>;
constexpr int tile_cost(int br_shift, int D) { return br_shift == 8 && D == 64 ? 5 : 1; }
// The cost of beginning a unit. Units of 256 rows: three tiles of two halves (2 and 4: up to 3 %
// slower). Few rows, in tiles: e4m3 tiles are short, 3 against 0 takes 256 sequences of about 1000
// keys from 157 to 127 us, 5 of 47500 from 49.5 to 48.0. 64 columns: 64 sequences of 2000 keys and
// 8 kv heads 67.4, 63.7, 64.7 us at 0, 1, 2. bf16 rows of 256 bytes: the ring hides it (194.2
// against 200.5 us for 64 long sequences), but with fewer units than CTAs (`few`), where a CTA of
// two pieces ends last (12.4 against 10.9 us for 3 sequences). 16 rows: twice the work at either
// end of a piece and a shorter ring; 0, 2, 4, 6, 9: 131, 122, 119, 121, 125 us for 128 sequences of
// 2200 keys, 16 + 4 heads, 4 tokens each, in bf16, and 119, 123, 118, 117, 121 in e4m3.
constexpr int unit_cost(int br_shift, int D, bool fp8, bool few) {
  return br_shift == 8   ? 3 * tile_cost(8, D)
         : br_shift == 4 ? (fp8 ? 6 : 4)
         : fp8           ? 3
         : few           ? 2
         : D == 64       ? 1
                         : 0;
}

// An upper bound on the length of a launch's line: T tokens in S sequences of at most `cap` keys.
inline double line_bound(int br_shift, int G, int hkv, int D, bool fp8, double T, double S,
                         double cap) {
  return hkv * (T * G / (1 << br_shift) + S) *
         ((cap / kAttnTK + 1) * tile_cost(br_shift, D) + unit_cost(br_shift, D, fp8, true));
}

// log2 of the rows per unit that a batch runs in, 0 when no line fits an int. By the query rows
// per sequence and kv head, on average (the lengths are on the device); any launch is right for
// any batch. 32 sequences of 2200 keys, 8 kv heads of 4 query heads, 1, 4, 6 and 8 tokens each: 52,
// 61, 125, 132 us in units of 8 and 16 rows, 60, 61, 61, 62 on the tensor cores (units of 256);
// 5 sequences of 47500 keys and 16 query heads a kv head in e4m3 73 and 88. A line that is too
// long in the units chosen may still fit in those of 8 rows, whose costs are the lowest (heads of
// 64, block tables of 500,000 positions and more).
inline int unit_shift(int G, int hkv, int D, bool fp8, int T, int S, double cap) {
  const long long rows = (long long)T * G;
  const int first = rows <= 8ll * S ? 3 : rows <= 16ll * S ? 4 : 8;
  if (cap > 1 << 30) cap = 1 << 30;  // as checked_seq cuts lengths
  auto fits = [&](int shift) {
    return line_bound(shift, G, hkv, D, fp8, T, S, cap) < 2147483640.0;
  };
  return fits(first) ? first : fits(3) ? 3 : 0;
}

}  // namespace gbmoe
