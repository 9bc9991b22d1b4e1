// How decode attention over the eight-bit cache cuts the blocks of all (sequence, kv head) pairs
// into pieces: their borders, what of a pair lies in a piece, and the parts' slots.  Every CTA
// and every join work it out for themselves, so it stands here once, in whole numbers, and builds
// for the host, where a test goes through it.
#pragma once

#ifndef EE_HD
#ifdef __CUDACC__
#define EE_HD __host__ __device__ __forceinline__
#else
#define EE_HD inline
#endif
#endif

namespace ee {

// A CTA's share of a pair: blocks first .. first + blocks - 1, `have` tokens in them.
struct Share {
  int s, g, first, blocks, have;
  int slot;  // of its part in the scratch; -1: the whole pair
};

// A pair of n blocks has the places [x, x + start + n): its first block stands at x, block b at
// x + start + b.  With start = 0 a pair's places are rounded up to whole pieces.  Pairs stand in
// the order of sequences, kv heads within.
struct DecodePieces {
  static constexpr int kStart = 6;  // a pair's beginning takes a CTA as long as so many blocks
  int hkv, start, each;             // places of a piece

  EE_HD static int smaller(int a, int b) { return a < b ? a : b; }
  EE_HD static int larger(int a, int b) { return a > b ? a : b; }
  // Even pieces of all pairs' blocks, `least` places at least.  (A piece of kStart + 1 places has a
  // block of every pair that it lies within.)
  EE_HD void cut(int hkv_, int blocks, int pairs, int pieces, int least) {
    hkv = hkv_;
    start = kStart;
    each = larger(larger(least, kStart + 1), (hkv * (blocks + kStart * pairs) + pieces - 1) / pieces);
  }
  // Pieces of c blocks, pairs cut by themselves, if that takes no more of them: `parts` of one kv head.
  EE_HD void cut_alone(int c, int parts, int pieces) {
    if (start && c <= each && hkv * parts <= pieces) {
      start = 0;
      each = c;
    }
  }
  EE_HD int places(int blocks) const {
    return start ? (blocks > 0 ? start + blocks : 0) : (blocks + each - 1) / each * each;
  }
  // The first block of a pair of n at x that stands at place c or behind it.
  EE_HD int block_at(int c, int x, int n) const { return c <= x ? 0 : smaller(n, larger(1, c - x - start)); }

  // What the piece [begin, end) of CTA `me` has of the pair that holds place *c, of sequence s of n
  // tokens, whose first pair stands at `base`.  False: none of it; *c: behind the pair.  A piece has at most two
  // parts, of its first pair and of its last.
  EE_HD bool share(int* c, int me, int begin, int end, int s, int base, int n, Share* w) const {
    const int from = *c, nb = (n + 15) >> 4, len = places(nb);
    w->s = s;
    w->g = (from - base) / len;
    const int x = base + w->g * len;
    *c = x + len;
    w->first = block_at(begin, x, nb);
    w->blocks = block_at(end, x, nb) - w->first;
    w->have = smaller(n - w->first * 16, w->blocks * 16);
    w->slot = w->blocks < nb ? 2 * me + (from > begin) : -1;
    return w->blocks > 0;
  }

  // The parts of a pair of nb blocks at x, for the join: of `count` CTAs from `first` on, if that
  // is more than one.
  struct Parts {
    int first, count, late;
    // The first CTA has the pair as its last one, unless it begins with it.
    EE_HD int slot(int k) const { return 2 * (first + k) + (k == 0 ? late : 0); }
  };
  EE_HD Parts parts(int x, int nb) const {
    Parts r;
    r.first = x / each;
    r.count = nb == 0 ? 0 : (nb == 1 ? x : x + start + nb - 1) / each - r.first + 1;
    r.late = x > r.first * each;
    return r;
  }
};

}  // namespace ee
