// How decode attention behind a shared prefix divides its work: which CTAs take the prefix and
// which the sequences' own blocks, the borders of their pieces, and the slots of their parts.
//
// Every CTA works this out for itself, and the join once more for each row, from lengths on the
// device: they have to agree to the last place.  So it is in whole numbers alone, in one
// place, and builds for the host, where a test goes through it.
#pragma once

#include <stdint.h>

#ifndef EE_HD
#ifdef __CUDACC__
#define EE_HD __host__ __device__ __forceinline__
#else
#define EE_HD inline
#endif
#endif

namespace ee {

constexpr int kKeys = 128;  // of a tile, eight blocks
constexpr int kMaxPieces = 160;
constexpr int kMostPlaces = (1 << 24) - 1;  // of an estimate
// Times in 200 cycles, by which the CTAs are shared out: a prefix tile, a unit's first loads and
// its part's way out, a CTA's beginning; a pair's beginning in blocks, a stream's beginning.  In eighths
// of that an own block of a stream, and 2^-19 of them a block, for each of hd, where all SMs together
// are as fast as the memory.
constexpr int kWideCost = 24, kNarrowCost = 12, kWideStart = 25, kNarrowStart = 18, kPrefixBegin = 85;
constexpr int kOwnStart = 11, kOwnBegin = 50, kOwnCost = 17, kOwnShare = 413;

// A prefix unit's share of a CTA: `tiles` key tiles, `have` tokens in them, from block `first`
// on.
struct Work {
  int kind;  // 0: no more, 1: narrow, 2: wide
  int s, g, first, tiles, have, rows;
  int64_t slot;  // of its part
  uint32_t par;  // bit i: of place i's tiles before this unit, odd or even
  int start;     // of a wide unit in the ring
};

// A stream's share of a (sequence, kv head): `blocks` from block `first` of table row `row` on,
// `have` tokens in them.
struct Own {
  int s, g, row, first, blocks, have;  // s = -1: no more
  int64_t slot;
};

// The scratch: parts of the prefix in slots of prefix_rows() rows each, then those of the own
// blocks in slots of G rows.
EE_HD int prefix_rows(int batch, int G) { return batch * G < 256 ? batch * G : 256; }
EE_HD int64_t prefix_slots(int batch, int G, int hkv, int prefix) {
  return prefix > 0 ? (int64_t)(batch * G + 255) / 256 * hkv + kMaxPieces : 0;
}
EE_HD int64_t own_slots(int batch, int hkv) { return (int64_t)batch * hkv + 2 * kMaxPieces; }
EE_HD int64_t scratch_rows(int batch, int G, int hkv, int prefix) {
  return prefix_slots(batch, G, hkv, prefix) * prefix_rows(batch, G) + own_slots(batch, hkv) * G;
}

// Where the pieces' borders lie.  A prefix unit of n tiles has the places [x, x + start + n
// cost): its first tile stands at x, tile k at x + start + k cost.  A pair's n own blocks
// likewise, with kOwnStart and cost 1; pairs stand in the order of sequences, kv heads within.
template <int G>
struct Pieces {
  int hkv, batch, prefix;
  int pre;                       // the prefix's blocks, 0 where no sequence sees it whole
  int pre_end, own_end;          // places
  int n_pre, each_pre, each_own;  // CTAs for the prefix; places of a CTA's piece, and of a stream's

  EE_HD static int least(int a, int b) { return a < b ? a : b; }
  EE_HD static int most(int a, int b) { return a > b ? a : b; }
  EE_HD static int places(int n, int start, int cost) { return n > 0 ? start + n * cost : 0; }
  EE_HD static int above(int a, int b) { return (a + b - 1) / b; }
  EE_HD int tiles() const { return (pre + 7) >> 3; }
  EE_HD int rows_of(int rt) const { return least(256, batch * G - rt * 256); }
  EE_HD int start_of(int rt) const { return rows_of(rt) > 128 ? kWideStart : kNarrowStart; }
  EE_HD int cost_of(int rt) const { return rows_of(rt) > 128 ? kWideCost : kNarrowCost; }
  EE_HD int pre_places(int rt) const { return rows_of(rt) > 0 ? places(tiles(), start_of(rt), cost_of(rt)) : 0; }
  EE_HD int first_own(int n) const { return pre > 0 && n >= pre * 16 ? pre : 0; }  // block
  EE_HD int own_blocks(int n) const { return ((n + 15) >> 4) - first_own(n); }
  EE_HD int own_places(int n) const { return places(own_blocks(n), kOwnStart, 1); }

  EE_HD void init(int hkv_, int batch_, int prefix_, bool whole) {
    hkv = hkv_;
    batch = batch_;
    prefix = prefix_;
    // who does not see the prefix whole has all its blocks to itself
    pre = whole ? prefix >> 4 : 0;
    pre_end = hkv * (pre_places(0) + pre_places(1));
  }
  EE_HD int piece_pre(int n) const { return most(kNarrowCost, above(pre_end, n)); }
  EE_HD int piece_own(int streams) const { return most(kOwnStart + 1, above(own_end, streams)); }
  // The i-th of 32 numbers of prefix CTAs, and the time of the slower kind with it before the number.
  EE_HD uint32_t estimate(int i, int ctas, int pairs, int head_dim) const {
    const int n = 1 + i * most(0, ctas - 2) / 31;
    const int a = 8 * (kPrefixBegin + piece_pre(n));
    const int64_t all = (int64_t)(own_end - kOwnStart * pairs) * head_dim * kOwnShare >> 19;
    const int64_t b = 8 * kOwnBegin + most(kOwnCost * piece_own(2 * most(1, ctas - n)), (int)(all < kMostPlaces ? all : kMostPlaces));
    return (uint32_t)(b < a ? a : b < kMostPlaces ? b : kMostPlaces) << 8 | (uint32_t)n;
  }
  // n: the number of prefix CTAs with the least estimate, where there is work of both kinds.
  EE_HD void share_out(int ctas, int n) {
    static_assert(kMaxPieces < 256, "a number of CTAs in eight bits");
    n_pre = pre_end == 0 ? 0 : own_end == 0 ? ctas : n;
    each_pre = piece_pre(most(1, n_pre));
    each_own = piece_own(2 * most(1, ctas - n_pre));
  }

  // The first tile (or block) of a unit at x that stands at place c or behind it.
  EE_HD static int item_at(int c, int x, int n, int start, int cost) {
    return c <= x ? 0 : least(n, most(1, (c - x - start + cost - 1) / cost));
  }
  EE_HD int64_t pre_slot(int rt, int g, int me) const { return rt * hkv + g + me; }
  EE_HD int64_t own_slot(int s, int g, int me) const { return (int64_t)s * hkv + g + me; }

  // The share of CTA `me` of the prefix unit that holds place *c, or of the next one that has any;
  // *c: behind the unit.
  EE_HD Work prefix_at(int* c, int me) const {
    Work w;
    const int begin = me * each_pre, stop = least(pre_end, begin + each_pre);
    w.kind = w.tiles = 0;
    while (*c < stop) {
      const int rt = *c < hkv * pre_places(0) ? 0 : 1, c0 = rt * hkv * pre_places(0), len = pre_places(rt);
      w.g = (*c - c0) / len;
      const int x = c0 + w.g * len;
      *c = x + len;
      const int k0 = item_at(begin, x, tiles(), start_of(rt), cost_of(rt)), k1 = item_at(stop, x, tiles(), start_of(rt), cost_of(rt));
      if (k1 == k0) continue;
      w.rows = rows_of(rt);
      w.kind = w.rows > 128 ? 2 : 1;
      w.s = rt * 256 / G;
      w.slot = pre_slot(rt, w.g, me);
      w.first = k0 * 8;
      w.have = least(pre * 16, k1 * kKeys) - k0 * kKeys;
      w.tiles = k1 - k0;
      break;
    }
    return w;
  }
  // The share of stream `me` of the pair that holds place *c: sequence s of n tokens, whose first
  // pair stands at `base`.  False: none of it; *c: behind the pair.
  EE_HD bool own_at(int* c, int me, int s, int base, int n, Own* w) const {
    const int begin = me * each_own, stop = least(own_end, begin + each_own);
    const int len = own_places(n), from = first_own(n), nb = own_blocks(n);
    w->s = s;
    w->g = (*c - base) / len;
    const int x = base + w->g * len;
    *c = x + len;
    const int k0 = item_at(begin, x, nb, kOwnStart, 1), k1 = item_at(stop, x, nb, kOwnStart, 1);
    w->row = prefix > 0 && from == 0 ? 0 : s;  // who ends within the prefix has its blocks
    w->first = from + k0;
    w->blocks = k1 - k0;
    w->have = least(n - w->first * 16, w->blocks * 16);
    w->slot = own_slot(s, w->g, me);
    return k1 > k0;
  }

  // What the join adds: the pieces that a unit's tiles (a pair's blocks) lie in, and whether piece i
  // has any of them.
  struct Range {
    int x, n, start, cost, each, first, last;  // pieces first .. last
    EE_HD bool has(int i) const {
      return item_at((i + 1) * each, x, n, start, cost) > item_at(i * each, x, n, start, cost);
    }
  };
  EE_HD static Range range(int x, int n, int start, int cost, int each) {
    return Range{x, n, start, cost, each, x / each, (n == 1 ? x : x + start + (n - 1) * cost) / each};
  }
  EE_HD Range prefix_range(int rt, int g) const {
    return range(rt * hkv * pre_places(0) + g * pre_places(rt), tiles(), start_of(rt), cost_of(rt), each_pre);
  }
  EE_HD Range own_range(int base, int g, int n) const {
    return range(base + g * own_places(n), own_blocks(n), kOwnStart, 1, each_own);
  }
};

}  // namespace ee
