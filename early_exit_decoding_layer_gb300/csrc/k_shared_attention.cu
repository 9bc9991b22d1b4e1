// Decode attention of a batch whose sequences begin with the same blocks, on the tensor
// cores (tcgen05.mma, fp32 accumulators in tensor memory).
//
// The shared blocks are read once for all rows: of a kv head there are B G of them
// (every sequence's query heads), 128 to an M tile, and what a decode step is bound
// by, bytes, becomes flops there.  The blocks behind the prefix have G rows each to read
// them, and are bound by bytes.  So the CTAs, one to an SM, are of two kinds that run side by
// side, as many of each as the lengths (which are on the device) make the times even.
//
// Prefix: S = Q K^T with 128 rows to an M tile, a unit being (row tile, kv head) and a CTA's
// piece a share of the units' key tiles.  Two streams, each with a softmax warpgroup; while
// one is busy with its probabilities the tensor core works for the other:
//   wide (a unit of 129 to 256 rows)  each stream has 128 rows, both see every key tile
//   narrow (up to 128 rows)  both have the same rows, and every second key tile;
//                           their results are added before they go out
//   warps 4t .. 4t + 3   a thread per row: S_t to registers, running maximum and sum,
//                        P_t = exp2(c S - c m) over S_t's columns, in two halves of 64
//                        keys, so that half of P V is done before the other is there
//   warp 9 (one thread)  the products, O_t += P_t V_j and S_t = Q K_j'^T; in narrow units
//                        stream 0's
//   warp 10              narrow: stream 1's products.  wide: waits for K and V tiles in warp
//                        9's place, which has none of the tensor core's time to lose, and
//                        frees those that are done with
//   warp 8               Q, K and V by TMA, a box per 16-slot block, into a ring
//
// Own blocks: S^T = K Q^T and O^T = V^T P with the cache as the big operand, 128 tokens x 16
// columns, a unit being (sequence, kv head).  With rows as M as above, G of 128 would be
// used and a tile take a thread 128 exponentials in a row: 3600 cycles instead of 1300.
// Two streams that know nothing of each other, each with a piece of all units' blocks:
//   warps 4t .. 4t + 3   a thread per token: scores, maximum, P into shared memory
//   warps 9, 10          (one thread) the products of stream 0 and 1
//   warps 8, 11          Q, K and V of stream 0 and 1
//
// A unit's result comes in parts, (O, m, l) in fp32 in the scratch; k_join adds each row's
// parts in the order of the pieces.  Maxima may lag behind by up to 8 (in log2), so
// that O is rarely rescaled.
//
// Probabilities go to the product as two fp16 terms, P = P_hi + P_lo: 22 bits, down to 2^-32 of
// a row's largest (they are lifted by 2^7, and 2^15 at most).  The second term is more MMAs with
// the same V in prefix units, and free in own blocks, whose products have 16 columns for G <= 8
// heads.  Rounded to fp16 once, each would be off by up to 2^-12, which in a mean of V is as much as
// the result's own rounding.
//
// Measured: 64 sequences behind 15000 tokens (64 query heads on 8 of 128) 73 us, 450 TFLOP/s and
// 3.2 TB/s; a wide step takes 4900 cycles, of which the tensor core is busy with 3400 (P_lo's MMAs
// 1000 of them; without them 3350 and 64 us).  32 behind 2048 (32 on 8) 16.7 us, 4 behind 512 (32
// on 8 of 64) 10.4 us: a CTA's beginning (4.5 us), few steps, and the join (2 to 3 us).
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "ee_decode_plan.cuh"
#include "ee_shared_plan.cuh"
#include "ee_tcgen05.cuh"

namespace ee {
namespace {

constexpr int kThreads = 384;  // two softmax warpgroups, TMA, two for MMA, units
// P is 2^kLift at the maximum, 2^(kLift + kLag) at most.
constexpr float kLift = 7.0f, kLag = 8.0f;

template <int HD>
struct Shape {
  static constexpr int H = HD / 64;                // 64-column halves
  static constexpr uint32_t kTile = 128 * HD * 2;  // a Q, K or V tile
  static constexpr uint32_t kHalf = 128 * 128;     // a 64-column half of Q's
  static constexpr uint32_t kRows8 = H * 1024;     // 8 tokens of K or V: [half][8][64]
  static constexpr int NST = HD == 128 ? 5 : 9;    // ring tiles: as many as fit
  static constexpr int D = (NST - 1) / 4;          // K tiles, and V tiles, of a stream in narrow units
  // own blocks: each stream's ring of K and V tiles, Q twice (16 rows of 128 bytes for every 64
  // columns), P (a row of 32 bytes for every token)
  static constexpr int NR = HD == 128 ? 3 : 6;
  static constexpr uint32_t kQ = H * 2048, kP = kKeys * 32;
  static constexpr uint32_t oQ = NR * kTile, oP = oQ + 2 * kQ, kStream = oP + kP;
  static_assert(kStream % 1024 == 0, "both streams' tiles are aligned");
  static constexpr size_t kSmem = 1024 + ((2 + NST) * kTile > 2 * kStream ? (2 + NST) * kTile : 2 * kStream);
};

struct Maps {
  CUtensorMap q, q1, k, v;  // q1: the rows of one sequence
};

// The parts in the scratch, rows of O and of (m, l).  First the prefix's, a slot of
// prefix_rows() rows each, with O as [hd / 8][rows][8]: rows next to each other, a thread's 32
// bytes each, are stored in one go.  Then the own blocks', G rows a slot.
struct Scratch {
  float *o, *ml;
};

// The pieces (ee_shared_plan.cuh), from lengths on the device: two sequences per lane, the whole
// warp.
template <int G>
struct Plan : Pieces<G> {
  using P = Pieces<G>;
  int tokens[2], base[2], size[2];  // of sequences lane and lane + 32: their own blocks' places, and those before them

  EE_DEV void init(const DecodeParams& p, int ctas) {
    static_assert(EE_MAX_BATCH <= 64, "two sequences per lane");
    static_assert((kOwnStart + kCacheMaxCtx / 16) * 32 < 1 << 16, "two sums in a word");
    const int lane = threadIdx.x & 31;
    int at[2];  // both loads before either is waited for
#pragma unroll
    for (int u = 0; u < 2; ++u) at[u] = lane + 32 * u < p.batch ? p.pos[lane + 32 * u] : -1;
#pragma unroll
    for (int u = 0; u < 2; ++u) tokens[u] = checked_length(at[u] == INT32_MAX ? at[u] : at[u] + 1, p.c.max_ctx, p.c.err);
    // the prefix is read if a sequence sees it whole
    P::init(p.c.n_kv_heads, p.batch, p.prefix, __any_sync(0xffffffffu, max(tokens[0], tokens[1]) >= p.prefix));
#pragma unroll
    for (int u = 0; u < 2; ++u) size[u] = P::own_places(tokens[u]);
    const uint32_t mine = (uint32_t)size[0] | (uint32_t)size[1] << 16;
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
    sum -= mine;
    base[0] = (int)(sum & 0xffffu);
    base[1] = (int)(all & 0xffffu) + (int)(sum >> 16);
    P::own_end = P::hkv * ((int)(all & 0xffffu) + (int)(all >> 16));
    int n = 0;
    if (P::pre_end > 0 && P::own_end > 0) {
      const int pairs = P::hkv * (__popc(__ballot_sync(0xffffffffu, size[0] > 0)) + __popc(__ballot_sync(0xffffffffu, size[1] > 0)));
      n = (int)(__reduce_min_sync(0xffffffffu, P::estimate(lane, ctas, pairs, p.c.head_dim)) & 255u);
    }
    P::share_out(ctas, n);
  }
  EE_DEV int of(const int (&a)[2], int s) const { return s < 32 ? __shfl_sync(0xffffffffu, a[0], s) : __shfl_sync(0xffffffffu, a[1], s - 32); }

  // The share of stream `me` of the pair that holds place *c, or of the next one that has any;
  // *c: behind the pair.
  EE_DEV Own own_at(int* c, int me) const {
    Own w;
    const int hkv = P::hkv, stop = min(P::own_end, (me + 1) * P::each_own);
    for (;;) {
      w.s = -1;
      w.blocks = 0;
      if (*c >= stop) return w;
      const unsigned lo = __ballot_sync(0xffffffffu, *c >= base[0] * hkv && *c < (base[0] + size[0]) * hkv);
      const unsigned hi = __ballot_sync(0xffffffffu, *c >= base[1] * hkv && *c < (base[1] + size[1]) * hkv);
      const int s = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
      if (P::own_at(c, me, s, of(base, s) * hkv, of(tokens, s), &w)) return w;
    }
  }
};

// Two probabilities as fp16 terms, the first in the low half.
EE_DEV void two_halves(float a, float b, uint32_t* hi, uint32_t* lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 r = __floats2half2_rn(a - f.x, b - f.y);
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&r);
}

template <int G>
EE_DEV Scratch scratch_of(const DecodeParams& p, bool own) {
  const int64_t rows = scratch_rows(p.batch, G, p.c.n_kv_heads, p.prefix);
  const int64_t before = own ? prefix_slots(p.batch, G, p.c.n_kv_heads, p.prefix) * prefix_rows(p.batch, G) : 0;
  Scratch r;
  r.o = reinterpret_cast<float*>(((uintptr_t)p.scratch + 31) & ~(uintptr_t)31);
  r.ml = r.o + rows * p.c.head_dim + before * 2;
  r.o += before * p.c.head_dim;
  return r;
}

// A stream of own blocks.
template <int HD, int G>
struct Stream {
  static constexpr int NR = Shape<HD>::NR;
  uint64_t full[NR], empty[NR], q_full[2], q_free[2], s_full[2], p_ready, o_done;  // Q by share & 1
  uint64_t drained;  // every MMA issued is over
  Ring<Own> shares;
  float red[4][G], sum[4][G];
};

template <int HD, int G>
struct Shared {
  static constexpr int NST = Shape<HD>::NST;
  uint64_t q_full[2], q_free[2], kv_full[NST], kv_empty[NST], s_full[2], p_ready[2][2], o_done[2];  // P in halves
  uint64_t drained[2];  // every MMA issued is over
  uint64_t both;        // narrow units: both streams' m, l and O are there; have been read
  Ring<Work> units;
  Stream<HD, G> own[2];
  bool prefix;  // this CTA has a piece of it
  uint32_t tmem;
};

// The CTA's two streams of own blocks, `first` and the next of all.
template <int HD, int G>
EE_DEV void own_blocks(const DecodeParams& p, const Maps& maps, float c, const Plan<G>& plan, Stream<HD, G>* streams, uint8_t* memory,
                       uint32_t tmem) {
  using S = Shape<HD>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x & 127;
  const int t = warp < 8 ? warp >> 2 : warp >= 10;  // the stream
  Stream<HD, G>& sh = streams[t];
  uint8_t* ring = memory + t * S::kStream;
  uint8_t *qs = ring + S::oQ, *ps = ring + S::oP;
  auto s_col = [&](int k) { return tmem + t * 64 + (k & 1) * 16; };
  auto o_col = [&](int r) { return tmem + t * 64 + 32 + (r & 1) * 16; };
  // Tile k's K is ring item 2 k, its V item 2 k + 1; tiles and shares count on.  After a wait
  // that gave up the softmax warps go on without waiting: they still meet each other.
  auto place = [&](int item) { return item % S::NR; };
  auto turn = [&](int item) { return item / S::NR; };
  bool ok = true;
  Own u;
  if (warp == 8 || warp == 11) {
    const int me = ((int)blockIdx.x - plan.n_pre) * 2 + t;
    int c0 = me * plan.each_own, n = 0;
    auto next = [&]() {
      const Own w = plan.own_at(&c0, me);
      ok = ok && sh.shares.put(n++, w, p.c.err);
      return w;
    };
    u = next();
    const uint64_t once = l2_evict_first_policy();
    int item = 0, r = 0;
    while (u.s >= 0 && ok) {
      const Own then = next();  // known before this one's last tile is issued
      if (!ok) break;
      const int32_t* table = p.c.table + (int64_t)u.row * p.c.table_stride + u.first;
      int ids = lane < u.blocks ? table[lane] : 0;  // 32 at a time
      if (r >= 2) ok = warp_wait(&sh.q_free[r & 1], (r / 2 - 1) & 1, p.c.err, DERR_EMPTY_WAIT);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.q_full[r & 1], G * HD * 2);
        for (int h = 0; h < S::H; ++h)
          tma_load_3d(smem_addr(qs + (r & 1) * S::kQ + h * 2048), &maps.q1, h * 64, u.g * G, u.s, &sh.q_full[r & 1]);
      }
      __syncwarp();
      ++r;
      for (int j = 0; j < u.blocks && ok; j += 8) {
        if (j > 0 && (j & 31) == 0) ids = j + lane < u.blocks ? table[j + lane] : 0;
        const int here = min(8, u.blocks - j);
        int id = __shfl_sync(0xffffffffu, ids, (j & 31) + (lane & 7));
        if (id < 0 || id >= p.c.n_blocks) {
          if (lane < here) report(p.c.err, EE_DERR_BLOCK);
          id = 0;
        }
        for (int kv = 0; kv < 2; ++kv, ++item) {
          const int at = place(item);
          if (turn(item) > 0) ok = warp_wait(&sh.empty[at], (turn(item) - 1) & 1, p.c.err, DERR_EMPTY_WAIT);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[at], (uint32_t)here * 16 * HD * 2);
          __syncwarp();
          if (lane < here)
            tma_stream_4d(smem_addr(ring + at * S::kTile + lane * 2 * S::kRows8), kv ? &maps.v : &maps.k, 0, 0, 0,
                          (id * p.c.n_kv_heads + u.g) * 2, &sh.full[at], once);
        }
      }
      u = then;
    }
    // Copies land before the CTA ends, whichever warp gave up (where none did, they have).
    for (int i = max(0, item - S::NR); i < item; ++i)
      mbar_wait_bounded(&sh.full[place(i)], (uint32_t)turn(i) & 1, p.c.err, DERR_DRAIN_WAIT);
    for (int i = max(0, r - 2); i < r; ++i) mbar_wait_bounded(&sh.q_full[i & 1], (i >> 1) & 1, p.c.err, DERR_DRAIN_WAIT);
  } else if (warp >= 9) {
    constexpr uint32_t id_s = instr_desc(0, 16, kKeys), id_o = instr_desc(0, 16, HD, true, true);
    auto there = [&](int item) { return mbar_test(&sh.full[place(item)], turn(item) & 1); };
    auto scores = [&](int k, int r, bool last) {  // of a tile of share r
      tc_fence_after();
      const uint64_t a = smem_desc_sw128(smem_addr(ring + place(2 * k) * S::kTile), S::kRows8),
                     b = smem_desc_sw128(smem_addr(qs + (r & 1) * S::kQ));
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        mma_f16(s_col(k), a + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), b + (((kk >> 2) * 2048 + (kk & 3) * 32) >> 4), id_s, kk > 0);
      mma_commit(&sh.s_full[k & 1]);
      mma_commit(&sh.empty[place(2 * k)]);
      if (last) mma_commit(&sh.q_free[r & 1]);
    };
    int k = 0;
    bool out = false;  // tile k's scores
    ok = sh.shares.get(0, &u, p.c.err);
    for (int r = 0; ok && u.s >= 0; ++r) {
      Own then;
      if (!(ok = sh.shares.get(r + 1, &then, p.c.err))) break;
      const int tiles = (u.blocks + 7) >> 3;
      if (lane == 0) {
        for (int j = 0; j < tiles && ok; ++j, ++k) {
          if (!out) {
            if (!(ok = mbar_wait_bounded(&sh.q_full[r & 1], (r >> 1) & 1, p.c.err, DERR_FULL_WAIT) &&
                       mbar_wait_bounded(&sh.full[place(2 * k)], turn(2 * k) & 1, p.c.err, DERR_FULL_WAIT)))
              break;
            scores(k, r, j + 1 == tiles);
          }
          // The next tile's scores as soon as it is there, of this share or of the next; but the
          // product with P does not wait for them: places of the ring are free behind it.
          const int rn = j + 1 < tiles ? r : r + 1;
          const bool more = j + 1 < tiles || then.s >= 0, last = j + 1 < tiles ? j + 2 == tiles : then.blocks <= 8;
          out = false;
          Patience patience;
          while (!(mbar_test(&sh.p_ready, k & 1) && there(2 * k + 1))) {
            if (more && !out && mbar_test(&sh.q_full[rn & 1], (rn >> 1) & 1) && there(2 * k + 2)) {
              scores(k + 1, rn, last);
              out = true;
            }
            if (patience.over(p.c.err, DERR_FULL_WAIT)) {
              ok = false;
              break;
            }
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t v = smem_desc_sw128_mn(smem_addr(ring + place(2 * k + 1) * S::kTile), 1024, S::kRows8),
                         x = smem_desc_rows<32>(smem_addr(ps), 256);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_f16(o_col(r), v + kk * (2 * S::kRows8 >> 4), x + kk * (512 >> 4), id_o, j > 0 || kk > 0);
          mma_commit(&sh.empty[place(2 * k + 1)]);
          mma_commit(&sh.o_done);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      k = __shfl_sync(0xffffffffu, k, 0);
      u = then;
    }
    if (lane == 0) {  // and so are the products, before tensor memory is given back
      mma_commit(&sh.drained);
      mbar_wait_bounded(&sh.drained, 0, p.c.err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else {
    const int w4 = warp & 3, bar = 1 + t;
    const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
    // M = 64: rows 16 w .. 16 w + 15 in the first lanes of warp w's part of tensor memory
    const int dim = HD == 128 ? tid : w4 * 16 + (lane & 15);
    const bool has_dim = HD == 128 || lane < 16;
    int k = 0;
    for (int r = 0;; ++r) {
      // the four warps go on together or not at all
      int go = sh.shares.get(r, &u, p.c.err) && u.s >= 0;
      asm volatile(
          "{ .reg .pred p, q; setp.ne.s32 p, %0, 0; barrier.cta.red.and.pred q, %1, 128, p; selp.s32 %0, 1, 0, q; }"
          : "+r"(go)
          : "r"(bar)
          : "memory");
      if (!go) break;
      const int tiles = (u.blocks + 7) >> 3;
      float m[G], l[G];  // m: kLift below the maximum
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.0f;
      }
#pragma unroll 1
      for (int j = 0; j < tiles; ++j, ++k) {
        if (ok) ok = warp_wait(&sh.s_full[k & 1], (k >> 1) & 1, p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        uint32_t v[16];
        tmem_ld16(s_col(k) + lane_base, v);
        tmem_wait_ld();
        tmem_pin<16>(v);
        const int left = u.have - j * kKeys;  // tokens from this tile on
        const bool live = tid < left;
        float z[G], a[G];
        int grow = 0;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          z[h] = live ? __uint_as_float(v[h]) * c : -INFINITY;
          grow |= z[h] - m[h] > kLift + kLag;
          a[h] = 1.0f;
        }
        asm volatile(
            "{ .reg .pred p, q; setp.ne.s32 p, %0, 0; barrier.cta.red.or.pred q, %1, 128, p; selp.s32 %0, 1, 0, q; }"
            : "+r"(grow)
            : "r"(bar)
            : "memory");
        if (grow) {  // the first tile, and rarely later
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float x = warp_max(z[h]);
            if (lane == 0) sh.red[w4][h] = x;
          }
          asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float mn = fmaxf(fmaxf(fmaxf(sh.red[0][h], sh.red[1][h]), fmaxf(sh.red[2][h], sh.red[3][h])) - kLift, m[h]);
            a[h] = m[h] == mn ? 1.0f : ex2(m[h] - mn);
            m[h] = mn;
            l[h] *= a[h];
          }
        }
        uint32_t hi[4] = {}, lo[4] = {};  // the token's row of P: columns h, and 8 + h
#pragma unroll
        for (int h = 0; h < G; h += 2) {
          float e[2] = {0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < (G == 1 ? 1 : 2); ++i) {
            e[i] = ex2(z[h + i] - (m[h + i] == -INFINITY ? 0.0f : m[h + i]));
            l[h + i] += e[i];
          }
          two_halves(e[0], e[1], &hi[h >> 1], &lo[h >> 1]);
        }
        // the product before has read P and is in O
        if (k > 0 && ok) ok = warp_wait(&sh.o_done, (k - 1) & 1, p.c.err, DERR_FULL_WAIT);
        *reinterpret_cast<uint4*>(ps + (tid >> 3) * 256 + row_chunk<32>(tid & 7, 0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(ps + (tid >> 3) * 256 + row_chunk<32>(tid & 7, 1)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (left < kKeys) {
          // slots behind the last token hold anything: their V becomes zero
          const int item = 2 * k + 1;
          if (ok) ok = warp_wait(&sh.full[place(item)], turn(item) & 1, p.c.err, DERR_FULL_WAIT);
          uint8_t* tile = ring + place(item) * S::kTile;
          for (int i = left * 8 + tid; i < kKeys * 8; i += 128)
#pragma unroll
            for (int half = 0; half < S::H; ++half)
              *reinterpret_cast<uint4*>(tile + (i >> 6) * S::kRows8 + half * 1024 + (i & 63) * 16) = make_uint4(0, 0, 0, 0);
        }
        if (grow && j > 0) {
          tc_fence_after();
          uint32_t o[16];
          tmem_ld16(o_col(r) + lane_base, o);
          tmem_wait_ld();
          tmem_pin<16>(o);
#pragma unroll
          for (int h = 0; h < G; ++h) {
            o[h] = __float_as_uint(__uint_as_float(o[h]) * a[h]);
            o[8 + h] = __float_as_uint(__uint_as_float(o[8 + h]) * a[h]);
          }
          tmem_st16(o_col(r) + lane_base, o);
          tmem_wait_st();
        }
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&sh.p_ready);
      }
      // the share's end: l of all warps, O of this thread's dim
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float x = warp_sum(l[h]);
        if (lane == 0) sh.sum[w4][h] = x;
      }
      if (ok) ok = warp_wait(&sh.o_done, (k - 1) & 1, p.c.err, DERR_FULL_WAIT);
      tc_fence_after();
      uint32_t o[16];
      tmem_ld16(o_col(r) + lane_base, o);
      asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
      tmem_wait_ld();
      tmem_pin<16>(o);
      const Scratch to = scratch_of<G>(p, true);
#pragma unroll
      for (int h = 0; h < G; ++h)
        if (has_dim) to.o[(u.slot * G + h) * HD + dim] = __uint_as_float(o[h]) + __uint_as_float(o[8 + h]);
#pragma unroll
      for (int h = 0; h < G; ++h)
        if (tid == h)
          *reinterpret_cast<float2*>(to.ml + (u.slot * G + h) * 2) =
              make_float2(m[h], (sh.sum[0][h] + sh.sum[1][h]) + (sh.sum[2][h] + sh.sum[3][h]));
      // sum is read before the next share's is written: its first tile's barrier is between
      tc_fence_before();
    }
  }
  if (!ok) __nanosleep(1000000);  // what this CTA no longer waited for may be on its way
}

template <int HD, int G>
__global__ void __launch_bounds__(kThreads, 1)
    k_shared_attention(const DecodeParams p, const __grid_constant__ Maps maps, const float c) {
  using S = Shape<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<HD, G> sh;
  uint8_t* tiles = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dep_launch();
  // The loads begin before anything else is ready: their warps make the barriers, and do not
  // wait for the others.
  const bool loads = warp == 8 || warp == 11;
  if (loads) {
    Stream<HD, G>& own = sh.own[warp == 11];
    if (lane < S::NR) {
      mbar_init(&own.full[lane], 1);
      mbar_init(&own.empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&own.q_full[lane], 1);
      mbar_init(&own.q_free[lane], 1);
      mbar_init(&own.s_full[lane], 1);
    }
    own.shares.init(5);  // four softmax warps and the one that issues
    if (lane == 0) {
      mbar_init(&own.p_ready, 128);
      mbar_init(&own.o_done, 1);
      mbar_init(&own.drained, 1);
    }
    if (warp == 8) {
      sh.units.init(10);  // eight softmax warps and the two that issue
      if (lane < S::NST) {
        mbar_init(&sh.kv_full[lane], 1);
        mbar_init(&sh.kv_empty[lane], 1);
      }
      if (lane < 2) {
        mbar_init(&sh.s_full[lane], 1);
        mbar_init(&sh.p_ready[lane][0], 129);  // its warpgroup, and the tiles that the products need
        mbar_init(&sh.p_ready[lane][1], 128);
        mbar_init(&sh.q_full[lane], 1);
        mbar_init(&sh.q_free[lane], 1);  // the stream's last product with it
        mbar_init(&sh.o_done[lane], 1);
        mbar_init(&sh.drained[lane], 1);
      }
      if (lane == 0) mbar_init(&sh.both, 256);
    }
    fence_mbar_init();
    __syncwarp();
    asm volatile("bar.arrive 3, %0;" ::"n"(kThreads) : "memory");
  }
  Plan<G> plan;
  bool prefix;
  if (loads) {
    plan.init(p, gridDim.x);
    prefix = (int)blockIdx.x < plan.n_pre;
    if (warp == 8) {
      if (lane == 0) sh.prefix = prefix;
      __syncwarp();
      asm volatile("bar.arrive 4, %0;" ::"n"(kThreads - 32) : "memory");
    }
  } else {
    if (warp == 9) {
      tmem_alloc(&sh.tmem, 512);
      tc_fence_before();
    }
    asm volatile("bar.sync 3, %0;" ::"n"(kThreads) : "memory");
    tc_fence_after();
    asm volatile("bar.sync 4, %0;" ::"n"(kThreads - 32) : "memory");
    prefix = sh.prefix;
  }
  const uint32_t tmem = loads ? 0 : sh.tmem;
  const uint32_t q_s = smem_addr(tiles), kv_s = q_s + 2 * S::kTile;
  // tensor memory: S_t (128 columns; P_t over them, of 32 keys each the 16 of P_hi, then P_lo's), then O_t
  auto s_col = [&](int t) { return tmem + t * 128; };
  auto o_col = [&](int t) { return tmem + 256 + t * HD; };
  // Steps of stream t in a unit, and the key tile of step k.
  auto steps_of = [](const Work& u, int t) { return u.kind == 2 ? u.tiles : (u.tiles + 1 - t) >> 1; };
  auto tile_of = [](const Work& u, int t, int k) { return u.kind == 2 ? k : 2 * k + t; };
  // Places in the ring.  A wide unit's K and V follow each other through all of it.  In
  // narrow units each stream has places of its own: then a place's tiles are waited for by one
  // thread, one after another, and however far a stream falls behind, the other cannot take
  // a phase of its barriers for the next one.
  struct Place {
    int at;
    uint32_t phase;
  };
  auto narrow_place = [](const Work& u, int t, int k, int kv) {
    Place x;
    x.at = t * 2 * S::D + k % S::D * 2 + kv;
    x.phase = (u.par >> x.at ^ (uint32_t)(k / S::D)) & 1;
    return x;
  };
  auto wide_place = [](const Work& u, int j, int kv) {
    Place x;
    x.at = (u.start + 2 * j + kv) % S::NST;
    x.phase = (u.par >> x.at ^ (uint32_t)((2 * j + kv) / S::NST)) & 1;
    return x;
  };
  auto landed = [&](const Place& x) {
    const bool r = mbar_wait_bounded(&sh.kv_full[x.at], x.phase, p.c.err, DERR_FULL_WAIT);
    tc_fence_after();
    return r;
  };

  constexpr uint32_t id_qk = instr_desc(0, kKeys, 128), id_pv = instr_desc(0, HD, 128, true);
  const uint64_t q_desc = smem_desc_sw128(q_s), k_desc = smem_desc_sw128(kv_s, S::kRows8),
                 v_desc = smem_desc_sw128_mn(kv_s, 1024, S::kRows8);
  auto product_s = [&](int t, int at) {  // S_t = Q_t K at a place
    const uint64_t a = q_desc + t * (S::kTile >> 4), b = k_desc + at * (S::kTile >> 4);
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk)
      mma_f16(s_col(t), a + (((kk >> 2) * S::kHalf + (kk & 3) * 32) >> 4), b + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id_qk, kk > 0);
  };
  auto product_o = [&](int t, int h, int at, bool acc) {  // O_t (+)= half h of P_t, V at a place
    const uint64_t b = v_desc + at * (S::kTile >> 4);
#pragma unroll
    for (int kk = h * kKeys / 32; kk < (h + 1) * kKeys / 32; ++kk)
#pragma unroll
      for (int low = 0; low < 2; ++low)
        mma_f16_ta(o_col(t), s_col(t) + (kk >> 1) * 32 + low * 16 + (kk & 1) * 8, b + (kk * 2 * S::kRows8 >> 4), id_pv,
                   acc || kk > h * kKeys / 32 || low > 0);
  };

  if (!prefix) {
    own_blocks<HD, G>(p, maps, c, plan, sh.own, tiles, tmem);
  } else if (warp == 8) {
    // this CTA's next unit
    int c0 = blockIdx.x * plan.each_pre, start = 0, n = 0;
    uint32_t par = 0;
    bool ok = true;
    auto next_unit = [&]() {
      Work w = plan.prefix_at(&c0, blockIdx.x);
      w.par = par;
      w.start = start;
      if (w.kind == 2) {
#pragma unroll 1
        for (int x = 0; x < S::NST; ++x) {
          const int first = (x - start + S::NST) % S::NST;
          par ^= first < 2 * w.tiles ? (uint32_t)((2 * w.tiles - first + S::NST - 1) / S::NST & 1) << x : 0;
        }
        start = (start + 2 * w.tiles) % S::NST;
      } else {
#pragma unroll 1
        for (int x = 0; x < 4 * S::D; ++x) {
          const int first = x % (2 * S::D) / 2, n = steps_of(w, x / (2 * S::D));
          par ^= first < n ? (uint32_t)((n - first + S::D - 1) / S::D & 1) << x : 0;
        }
      }
      ok = ok && sh.units.put(n++, w, p.c.err);
      return w;
    };
    Work u = next_unit();
    const int b8 = lane & 7;
    int at0 = 0, ends[2] = {0, 0};  // the next place of a wide unit
    uint32_t loaded = 0;  // as Work's par, but for every tile
    for (; u.kind && ok; u = next_unit()) {
      const int nblk = (u.have + 15) >> 4;
      const int32_t* bt = p.c.table + u.first;  // the first row's
      auto block_id = [&](int j) {  // of block b8 of key tile j
        const int b = j * 8 + b8;
        int id = b < nblk ? bt[b] : 0;
        if (id < 0 || id >= p.c.n_blocks) {
          report(p.c.err, EE_DERR_BLOCK);
          id = 0;
        }
        return id;
      };
      // of the next two key tiles
      int id0 = block_id(0), id1 = block_id(1);
      at0 = u.start;
      // each stream's Q, in a wide unit its rows; q_free: the stream's products before have read theirs
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (steps_of(u, t) == 0) continue;
        if (ok && ends[t] > 0) ok = warp_wait(&sh.q_free[t], (ends[t] - 1) & 1, p.c.err, DERR_EMPTY_WAIT);
        if (!ok) break;
        ++ends[t];
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full[t], S::kTile);
          for (int h = 0; h < S::H; ++h)
            tma_load_3d(q_s + t * S::kTile + h * S::kHalf, &maps.q, h * 64, u.g * G, u.s + (u.kind == 2 ? t * (128 / G) : 0),
                        &sh.q_full[t]);
        }
        __syncwarp();
      }
      if (!ok) break;
      auto load = [&](int j, int kv, int id, int at) {
        const int here = min(8, nblk - j * 8);
        if (!ok || !(ok = warp_wait(&sh.kv_empty[at], (loaded >> at ^ 1) & 1, p.c.err, DERR_EMPTY_WAIT))) return;
        if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[at], (uint32_t)here * 16 * HD * 2);
        __syncwarp();
        if (lane < here)
          tma_load_4d(kv_s + at * S::kTile + lane * 2 * S::kRows8, kv ? &maps.v : &maps.k, 0, 0, 0,
                      (id * p.c.n_kv_heads + u.g) * 2, &sh.kv_full[at]);
        loaded ^= 1u << at;
      };
      for (int j = 0; j < u.tiles && ok; j += 2) {
        const int a = id0, b = id1;
        id0 = block_id(j + 2);
        id1 = block_id(j + 3);
        // wide: K and V of a tile, then of the next; narrow: K of both streams before their V,
        // whose places are free later
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          const bool wide = u.kind == 2;
          const int second = wide ? x >> 1 : x & 1, kv = wide ? x & 1 : x >> 1;
          if (j + second >= u.tiles) continue;
          load(j + second, kv, second ? b : a, wide ? at0 : narrow_place(u, second, j >> 1, kv).at);
          at0 = at0 + 1 == S::NST ? 0 : at0 + 1;
        }
      }
    }
    // Copies land before the CTA ends, whichever warp gave up (where none did, they have).
    for (int x = 0; x < S::NST; ++x) mbar_wait_bounded(&sh.kv_full[x], (loaded >> x ^ 1) & 1, p.c.err, DERR_DRAIN_WAIT);
    for (int t = 0; t < 2; ++t)
      if (ends[t] > 0) mbar_wait_bounded(&sh.q_full[t], (ends[t] - 1) & 1, p.c.err, DERR_DRAIN_WAIT);
  } else if (warp == 9 || warp == 10) {
    const int me = warp - 9;
    Work u;
    int steps[2] = {0, 0}, ends[2] = {0, 0};
    bool ok = true;
    for (int i = 0; ok && sh.units.get(i, &u, p.c.err) && u.kind; ++i) {
      const int nk = u.tiles;
      const bool wide = u.kind == 2;
      if (lane == 0) {
        auto q_there = [&](int t) {
          const bool r = mbar_wait_bounded(&sh.q_full[t], ends[t] & 1, p.c.err, DERR_FULL_WAIT);
          tc_fence_after();
          return r;
        };
        if (!wide) {
          // a stream by itself: each product as soon as its tile is there
          const int t = me, n = steps_of(u, t);
          auto scores = [&](int k) {
            const Place x = narrow_place(u, t, k, 0);
            if (!landed(x)) return false;
            product_s(t, x.at);
            mma_commit(&sh.s_full[t]);
            mma_commit(&sh.kv_empty[x.at]);
            return true;
          };
          if (ok && n > 0) ok = q_there(t) && scores(0);
          for (int k = 0; k < n && ok; ++k) {
            const Place v = narrow_place(u, t, k, 1);
            if (!(ok = landed(v))) break;
            mbar_arrive(&sh.p_ready[t][0]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (!ok || !(ok = mbar_wait_bounded(&sh.p_ready[t][h], steps[t] & 1, p.c.err, DERR_FULL_WAIT))) break;
              tc_fence_after();
              product_o(t, h, v.at, k > 0 || h > 0);
            }
            if (!ok) break;
            ++steps[t];
            mma_commit(&sh.kv_empty[v.at]);
            if (k + 1 < n) ok = scores(k + 1);
            else mma_commit(&sh.o_done[t]);
          }
        } else if (me == 0) {
          // One thread issues every product of both streams.  The tensor core takes an MMA
          // from it when it starts on it, so what the thread does between two products costs
          // the tensor core time: a step's O and next S products of a stream go out together, each
          // wait that can be left to another warp is, and commits are few.  The commit behind
          // S_t(j + 1) also says that O_t has P_t V_j.
          auto scores = [&](int t, int at) {
            product_s(t, at);
            mma_commit(&sh.s_full[t]);
          };
          int at = u.start;
          ok = ok && q_there(0) && q_there(1) && landed(wide_place(u, 0, 0));
          if (ok) {
            scores(0, at);
            scores(1, at);
          }
          for (int j = 0; j < nk && ok; ++j) {
            const int v = at + 1 == S::NST ? 0 : at + 1;
            at = v + 1 == S::NST ? 0 : v + 1;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              // P_t(j) is in tensor memory, V_j and K_{j + 1} have landed
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (!ok || !(ok = mbar_wait_bounded(&sh.p_ready[t][h], steps[t] & 1, p.c.err, DERR_FULL_WAIT))) break;
                tc_fence_after();
                product_o(t, h, v, j > 0 || h > 0);
              }
              if (!ok) break;
              ++steps[t];
              if (j + 1 < nk) scores(t, at);
              else mma_commit(&sh.o_done[t]);
            }
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (wide && me == 1) {
        // Waits for V_j and K_{j + 1} on behalf of the MMA thread (P_t(j)'s barriers count this
        // arrival too), and frees the tiles of products that are over: stream 1's come last in a
        // step.  (Its S_1(j + 1) waits for this warp, which so misses no phase of s_full.)
        for (int j = 0; j < nk && ok; ++j) {
          const Place v = wide_place(u, j, 1), k = wide_place(u, j + 1, 0);
          ok = warp_wait(&sh.kv_full[v.at], v.phase, p.c.err, DERR_FULL_WAIT);
          if (ok && j + 1 < nk) ok = warp_wait(&sh.kv_full[k.at], k.phase, p.c.err, DERR_FULL_WAIT);
          // one phase of p_ready per step: the one before has to be over
          if (ok && steps[0] + j > 0) ok = warp_wait(&sh.p_ready[0][0], (steps[0] + j - 1) & 1, p.c.err, DERR_FULL_WAIT);
          if (ok && lane == 0) mbar_arrive(&sh.p_ready[0][0]);
          if (ok) ok = warp_wait(&sh.s_full[1], (steps[1] + j) & 1, p.c.err, DERR_FULL_WAIT);
          if (ok && steps[1] + j > 0) ok = warp_wait(&sh.p_ready[1][0], (steps[1] + j - 1) & 1, p.c.err, DERR_FULL_WAIT);
          if (ok && lane == 0) {
            if (j > 0) mbar_arrive(&sh.kv_empty[wide_place(u, j - 1, 1).at]);
            mbar_arrive(&sh.kv_empty[wide_place(u, j, 0).at]);
            mbar_arrive(&sh.p_ready[1][0]);
          }
        }
        // and the last V's; so stream 1's products, which narrow units take from this warp, are over
        if (ok) ok = warp_wait(&sh.o_done[1], ends[1] & 1, p.c.err, DERR_FULL_WAIT);
        if (ok && lane == 0) mbar_arrive(&sh.kv_empty[wide_place(u, nk - 1, 1).at]);
      }
      ok = __all_sync(0xffffffffu, ok);
      // both warps count both streams' steps (those that they made themselves are counted)
      const int n0 = steps_of(u, 0), n1 = steps_of(u, 1);
      steps[0] = __shfl_sync(0xffffffffu, steps[0], 0) + (me == 0 ? 0 : n0);
      steps[1] = __shfl_sync(0xffffffffu, steps[1], 0) + ((wide ? me == 0 : me == 1) ? 0 : n1);
      ends[0] += n0 > 0;
      ends[1] += n1 > 0;
    }
    if (lane == 0) {  // and so are the products, before tensor memory is given back
      mma_commit(&sh.drained[me]);
      mbar_wait_bounded(&sh.drained[me], 0, p.c.err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else if (warp < 8) {
    const int t = warp >> 2, r = tid & 127;  // stream and row
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = s_col(t) + lane_base, o_at = o_col(t) + lane_base;
    Work u;
    int steps = 0, ends = 0;
    bool ok = true;
    for (int i = 0; ok && sh.units.get(i, &u, p.c.err) && u.kind; ++i) {
      const bool wide = u.kind == 2;
      const int n = steps_of(u, t);
      const int row = r + (wide ? t * 128 : 0);  // of the unit
      const bool busy = row - lane < u.rows;     // a row of this warp is the unit's
      float m = -INFINITY, l = 0.0f;  // m: c times the maximum, less kLift
      for (int k = 0; k < n && ok; ++k) {
        const int j = tile_of(u, t, k);
        if (!(ok = warp_wait(&sh.s_full[t], steps & 1, p.c.err, DERR_FULL_WAIT))) break;
        ++steps;
        tc_fence_after();
        if (r == 0 && k == n - 1) mbar_arrive(&sh.q_free[t]);  // the stream's last product with Q
        const int lim = u.have - j * kKeys;                 // keys of the tile that exist
        if (lim < kKeys) {
          // slots behind the last token hold anything: their V becomes zero
          const Place v = wide ? wide_place(u, j, 1) : narrow_place(u, t, k, 1);
          if (!(ok = warp_wait(&sh.kv_full[v.at], v.phase, p.c.err, DERR_FULL_WAIT))) break;
          uint8_t* tile = tiles + (2 + v.at) * S::kTile;
          for (int i = lim * 8 + r; i < kKeys * 8; i += 128)
#pragma unroll
            for (int half = 0; half < S::H; ++half)
              *reinterpret_cast<uint4*>(tile + (i >> 6) * S::kRows8 + half * 1024 + (i & 63) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async();
        }
        if (busy) {
          // In pieces of 32 keys, by loops that stay loops: a CTA has few steps, and its
          // instructions come from L2, or from DRAM behind everybody's tiles.  (All 128 keys in
          // registers: the first step took 9000 cycles, and 40000 beside CTAs that kept the memory
          // busy, now 4500; the others 1700, now 1900 to 2000.)
          uint32_t s[32];
          auto load = [&](int q) {
            tmem_ld32(s_at + 32 * q, s);
            tmem_wait_ld();
            tmem_pin<32>(s);
            if (lim < kKeys) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * q + i >= lim) s[i] = 0xff800000u;  // -inf
            }
          };
          float mt = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < kKeys / 32; ++q) {
            load(q);
            float mx[2] = {mt, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 4)
#pragma unroll
              for (int w = 0; w < 2; ++w)
                mx[w] = max3(mx[w], __uint_as_float(s[i + 2 * w]), __uint_as_float(s[i + 2 * w + 1]));
            mt = fmaxf(mx[0], mx[1]);
          }
          if (k == 0) {
            m = fmaf(mt, c, -kLift);
          } else if (__any_sync(0xffffffffu, row < u.rows && fmaf(mt, c, -m) > kLift + kLag)) {
            // some row's maximum has grown too far (rows that are not the unit's have no say: what
            // they hold depends on what was there before): this warp's rows of O and l go over to
            // the new maxima (O has every product before: S_t came after)
            const float mn = fmaxf(m, fmaf(mt, c, -kLift));
            const float a = m == mn ? 1.0f : ex2(m - mn);
            m = mn;
            l *= a;
#pragma unroll 1
            for (int i = 0; i < HD; i += 16) {
              uint32_t o[16];
              tmem_ld16(o_at + i, o);
              tmem_wait_ld();
              tmem_pin<16>(o);
#pragma unroll
              for (int w = 0; w < 16; ++w) o[w] = __float_as_uint(__uint_as_float(o[w]) * a);
              tmem_st16(o_at + i, o);
            }
          }
          // a row that has seen nothing yet has m = -inf: its P is 0
          const float ms = m == -INFINITY ? 0.0f : m;
          const uint64_t c2 = pack2(c, c), nm2 = pack2(-ms, -ms);
          uint64_t sum = 0;
#pragma unroll 1
          for (int q = 0; q < kKeys / 32; ++q) {
            load(q);
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x = unpack2(fma2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, nm2));
              const float e0 = ex2(x.x), e1 = ex2(x.y);
              sum = add2(sum, pack2(e0, e1));
              two_halves(e0, e1, &hi[i >> 1], &lo[i >> 1]);
            }
            tmem_st16(s_at + 32 * q, hi);
            tmem_st16(s_at + 32 * q + 16, lo);
            if (q == kKeys / 64 - 1) {  // the product with the first half while the second is made
              tmem_wait_st();
              tc_fence_before();
              mbar_arrive(&sh.p_ready[t][0]);
            }
          }
          const float2 st = unpack2(sum);
          l += st.x + st.y;
          tmem_wait_st();
        }
        if (!busy) mbar_arrive(&sh.p_ready[t][0]);
        tc_fence_before();
        mbar_arrive(&sh.p_ready[t][1]);
      }
      if (ok && n > 0) ok = warp_wait(&sh.o_done[t], ends & 1, p.c.err, DERR_FULL_WAIT);
      ends += n > 0;
      tc_fence_after();
      // the part: a thread has its row of O, 32 bytes a store.  Of a narrow unit with two streams each
      // warpgroup has half of the columns, of both: O = a_0 O_0 + a_1 O_1.  (A part of each
      // stream is twice as much to store, 5000 cycles instead of 2500, and to join: 32 sequences
      // behind 2048 19.7 us instead of 18.1.)
      const bool two = !wide && u.tiles > 1;
      float a0 = 1.0f, a1 = 0.0f;
      if (two) {
        // m and l, by unit & 1, stream and row, in the ring's place that narrow units (the last ones) leave free
        static_assert(4 * S::D < S::NST, "a free place");
        float2* ml = reinterpret_cast<float2*>(tiles + (1 + S::NST) * S::kTile) + (i & 1) * 256;
        ml[t * 128 + r] = make_float2(m, l);
        mbar_arrive(&sh.both);
        if (ok) ok = warp_wait(&sh.both, 0, p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        const float2 x = ml[r], y = ml[128 + r];
        m = fmaxf(x.x, y.x);
        a0 = x.x == m ? 1.0f : ex2(x.x - m);
        a1 = y.x == m ? 1.0f : ex2(y.x - m);
        l = fmaf(a0, x.y, a1 * y.y);
      }
      if (ok && n > 0 && busy) {
        const Scratch to = scratch_of<G>(p, false);
        const int R = prefix_rows(p.batch, G);
        float* o_to = to.o + u.slot * R * HD + row * 8;
        const int first = two ? t * (HD / 2) : 0, last = two ? first + HD / 2 : HD;
#pragma unroll 1
        for (int d = first; d < last; d += 32) {
          uint32_t o[32], other[32];
          tmem_ld32((two ? o_col(0) + lane_base : o_at) + d, o);
          if (two) tmem_ld32(o_col(1) + lane_base + d, other);
          tmem_wait_ld();
          tmem_pin<32>(o);
          if (two) {
            tmem_pin<32>(other);
#pragma unroll
            for (int w = 0; w < 32; ++w)
              o[w] = __float_as_uint(fmaf(a0, __uint_as_float(o[w]), a1 * __uint_as_float(other[w])));
          }
          if (row < u.rows) {
#pragma unroll
            for (int w = 0; w < 32; w += 8) st_global_v8(o_to + (d + w) / 8 * R * 8, o + w);
          }
        }
        if (row < u.rows && (!two || t == 0)) *reinterpret_cast<float2*>(to.ml + (u.slot * R + row) * 2) = make_float2(m, l);
      }
      if (two) {  // no product of the next unit's goes over what the other has not read
        tc_fence_before();
        mbar_arrive(&sh.both);
        if (ok) ok = warp_wait(&sh.both, 1, p.c.err, DERR_FULL_WAIT);
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// Adds the parts, of the prefix and of its own blocks, of every row.
template <int HD, int G, int J>
__global__ void __launch_bounds__(kJoinThreads) k_join(const DecodeParams p, const int ctas) {
  using Sum = Join<HD, J>;
  constexpr int P = Sum::P, U = Sum::kAtOnce, kStripes = Sum::kStripes;
  __shared__ int64_t ml_at[3 * kMaxPieces], o_at[3 * kMaxPieces];  // where head 0's parts are; -1: none
  __shared__ typename Sum::Stripes stripes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x / (p.n_heads / J), first = (blockIdx.x - s * (p.n_heads / J)) * J;  // its heads
  const int g = first / G, h = first % G + warp % J;
  Plan<G> plan;
  plan.init(p, ctas);
  const int n = plan.of(plan.tokens, s);
  const int own = plan.own_blocks(n);
  const int all = s * G, rt = all >> 8, row = all & 255, R = prefix_rows(p.batch, G);
  int n_pre = 0, count = 0;
  // the prefix's parts: one a piece
  if (plan.first_own(n) > 0) {
    const auto pieces = plan.prefix_range(rt, g);
    for (int i = pieces.first + tid; i <= pieces.last; i += kJoinThreads) {
      const int64_t slot = plan.pre_slot(rt, g, i);
      ml_at[i - pieces.first] = pieces.has(i) ? slot * R + row : -1;
      o_at[i - pieces.first] = slot * R * HD + row * 8;
    }
    n_pre = count = pieces.last - pieces.first + 1;
  }
  // and those of its own blocks
  if (own > 0) {
    const auto pieces = plan.own_range(plan.of(plan.base, s) * plan.hkv, g, n);
    for (int i = pieces.first + tid; i <= pieces.last; i += kJoinThreads) {
      const int64_t at = plan.own_slot(s, g, i) * G;
      ml_at[n_pre + i - pieces.first] = pieces.has(i) ? at : -1;
      o_at[n_pre + i - pieces.first] = at * HD;
    }
    count += pieces.last - pieces.first + 1;
  }
  // this lane's dims, lane * P and on: eight floats of a prefix row lie together
  const Scratch sp = scratch_of<G>(p, false), so = scratch_of<G>(p, true);
  const float *pre_o = sp.o + h * 8 + (int64_t)(lane * P / 8) * R * 8 + lane * P % 8, *own_o = so.o + h * HD + lane * P;
  grid_dep_wait();
  __syncthreads();
  Sum sum;
  for (int k0 = warp / J; k0 < count; k0 += kStripes * U) {
    float mk[U], lk[U], x[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + kStripes * u;
      const int64_t at = k < count ? ml_at[k] : -1;
      mk[u] = -INFINITY;
      lk[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < P; ++i) x[u][i] = 0.0f;
      if (at >= 0) {
        const float2 ml = *reinterpret_cast<const float2*>((k < n_pre ? sp.ml : so.ml) + (at + h) * 2);
        mk[u] = ml.x;
        lk[u] = ml.y;
        const float* from = (k < n_pre ? pre_o : own_o) + o_at[k];
        if constexpr (P == 4) *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(from);
        else *reinterpret_cast<float2*>(x[u]) = *reinterpret_cast<const float2*>(from);
      }
    }
    sum.add(mk, lk, x);
  }
  sum.finish(stripes, p.o + s * p.o_stride + first * HD);
}

template <int HD, int G>
cudaError_t launch_t(const DecodeParams& p, cudaStream_t st) {
  using S = Shape<HD>;
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_shared_attention<HD, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  Maps maps;
  const uint64_t qd[3] = {(uint64_t)HD, (uint64_t)p.n_heads, (uint64_t)p.batch};
  const uint64_t qs[2] = {(uint64_t)HD * 2, (uint64_t)p.q_stride * 2};
  const uint32_t many[3] = {64, (uint32_t)G, 128 / (uint32_t)G}, one[3] = {64, (uint32_t)G, 1};
  // a block of K or V at once, as groups of 8 rows: [group][half][8][64]
  const uint64_t cd[4] = {64, 8, (uint64_t)S::H, (uint64_t)p.c.n_blocks * p.c.n_kv_heads * 2},
                 cs[3] = {(uint64_t)HD * 2, 128, (uint64_t)HD * 16};
  const uint32_t cb[4] = {64, 8, (uint32_t)S::H, 2};
  if (!encode_tensor_map(&maps.q, false, 3, p.q, qd, qs, many) || !encode_tensor_map(&maps.q1, false, 3, p.q, qd, qs, one) || !encode_tensor_map(&maps.k, false, 4, p.c.k, cd, cs, cb) ||
      !encode_tensor_map(&maps.v, false, 4, p.c.v, cd, cs, cb))
    return cudaErrorInvalidValue;
  // a CTA per SM, but not many more than there are tiles
  const int64_t own = (int64_t)p.batch * p.c.n_kv_heads * ((p.c.max_ctx + kKeys - 1) / kKeys);
  const int64_t pre = (int64_t)((p.batch * G + 255) / 256) * p.c.n_kv_heads * ((p.prefix + kKeys - 1) / kKeys);
  const int ctas = (int)std::min<int64_t>(std::min(sms, kMaxPieces), own + pre);
  k_shared_attention<HD, G><<<ctas, kThreads, S::kSmem, st>>>(p, maps, make_exponent(HD).c);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return join_by_rows<G>(p.batch * p.n_heads, sms, [&](auto J) {
    return launch_join(k_join<HD, G, J.value>, p.batch * (p.n_heads / J.value), sms, S::kSmem, st, p, ctas);
  });
}

}  // namespace

cudaError_t launch_shared_attention(const DecodeParams& p, cudaStream_t st) {
  const int G = p.n_heads / p.c.n_kv_heads, hd = p.c.head_dim;
#define EE_SHARED_CASE(HD_, G_) \
  if (hd == HD_ && G == G_) return launch_t<HD_, G_>(p, st);
  EE_SHARED_CASE(64, 1)
  EE_SHARED_CASE(64, 2)
  EE_SHARED_CASE(64, 4)
  EE_SHARED_CASE(64, 8)
  EE_SHARED_CASE(128, 1)
  EE_SHARED_CASE(128, 2)
  EE_SHARED_CASE(128, 4)
  EE_SHARED_CASE(128, 8)
#undef EE_SHARED_CASE
  return cudaErrorInvalidValue;
}

size_t shared_attention_scratch(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t, int32_t prefix) {
  const int64_t rows = scratch_rows(batch, n_heads / n_kv_heads, n_kv_heads, prefix >= EE_KV_BLOCK ? prefix : 0);
  return (size_t)rows * (head_dim + 2) * 4 + 32;
}

}  // namespace ee
