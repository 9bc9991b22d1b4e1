// Decode attention over the eight-bit cache, on the tensor cores.
//
// One new token per sequence: K and V are read once for the G query heads of a kv
// head, so the bytes are the bound, and these are half of the fp16 cache's -- if the
// arithmetic keeps out of the way.  Turning codes into fp16 first would cost
// instructions for every byte; the MMAs take e4m3 as it is, with the cache as the big
// operand:
//   S = K_tile Q^T      128 tokens x N columns
//   O^T += V_tile^T X   head dims x N columns, K = 128 tokens
// Then Q and X have to be e4m3 too.  They go in as parts of four bits, three of Q and four of X,
//   x = a + 2^-5 b + 2^-10 c + 2^-15 d,
// each a column of its own (N = 4 G, at least 16).  A part's remainder is at most 2^-4 of it, and
// times 2^5 the next part is at most twice as large, so that it is off by 2^-4 of that again: three
// parts have 2^-14 of a value and so all bits of an fp16 query, four have 2^-19.  The parts end at
// 2^-9 in e4m3: queries are exact down to 2^-27 of a head's largest component (which is 2^7 or more),
// X is down to 2^-29 of its largest (2^4 or more).  The columns that this adds are free: the tensor
// core is at a few percent.
//
// The rows' scales are powers of two.  K's multiplies a score.  V's goes into the
// probability: with w_t = log2(e) z_t + e_t the product takes X_t = 2^(w_t - M), M a
// running maximum of w that may lag by 2^4, and the sum l adds X_t 2^-e_t, which is exact.
//
// A CTA has a piece of all blocks (ee_decode_plan.cuh), in tiles of eight blocks:
//   warps 0-3  a thread per token: scores, maximum, X into shared memory; then a
//              thread per head dim writes O, or a part of it to the scratch
//   warp 4     codes by TMA, one box a block (K and V lie side by side), and exponents,
//              into a ring
//   warp 5     (one thread) the MMAs, S a tile ahead of O
//   warps 6-7  the next pair's Q
// A second kernel joins the parts of pairs that several CTAs had a share of.
//
// Measured: 16 sequences of 16384 tokens (64 query heads on 8 of 128) 82 us, 6.3 TB/s; 32 of 257 to
// 2176 (32 on 8) 22 us, 3.5 TB/s, of which 8 us are a CTA's beginning and the join; one of 2113
// 8.1 us, one of 33 (4 on 2 of 64, no join) 5.3 us: latency.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "ee_decode_plan.cuh"
#include "ee_tcgen05.cuh"

namespace ee {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 128;  // per tile, eight blocks
constexpr int kMaxCtas = 3 * 160;
constexpr float kLift = 4.0f, kLag = 4.0f;  // X is 2^kLift at the maximum, 2^(kLift + kLag) at most

template <int HD, int G>
struct Layout {
  static constexpr int N = G == 8 ? 32 : 16;          // columns: part 0 of G heads, part 1, and so on
  static constexpr int kCtas = G == 8 ? 2 : 3;        // per SM
  static constexpr uint32_t kBlock = 32 * HD;         // K and V of a block: [2 groups][K, V][8][HD]
  static constexpr uint32_t kRows8 = 16 * HD;         // from 8 tokens to the next 8
  static constexpr uint32_t kTile = 8 * kBlock;
  static constexpr int NS = (HD == 64 ? 2 : 1) * (G == 8 ? 3 : 2);
  static constexpr uint32_t kQ = N * HD;              // rows of HD bytes
  static constexpr uint32_t kX = kTokens * 32;        // rows of 32 bytes, a token each
  static constexpr uint32_t oQ = NS * kTile, oX = oQ + 2 * kQ, oE = oX + kX;
  static constexpr size_t kSmem = 1024 + oE + NS * 256;
};

template <int HD, int G>
struct Shared {
  static constexpr int NS = Layout<HD, G>::NS;
  uint64_t full[NS], empty[NS], s_full[2], x_ready, o_done;
  uint64_t q_ready[2], q_free[2];  // by share & 1
  uint64_t drained;                // every MMA issued is over
  uint32_t tmem;
  Ring<Share> shares;
  float unscale[2][G], red[4][G], sum[4][G];
};

// What two e4m3 codes stand for.
EE_DEV float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// The parts of two values of at most 2^8.
template <int N>
EE_DEV void parts(float a, float b, uint32_t (&c)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    c[i] = to_e4m3x2(a, b);
    if (i < N - 1) {
      const float2 f = from_e4m3x2(c[i]);
      a = (a - f.x) * 32.0f;
      b = (b - f.y) * 32.0f;
    }
  }
}

// A value from the columns of its parts, the smallest first.
EE_DEV float joined(uint32_t a, uint32_t b, uint32_t c) {
  return fmaf(fmaf(__uint_as_float(c), 0x1p-5f, __uint_as_float(b)), 0x1p-5f, __uint_as_float(a));
}
EE_DEV float joined(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return joined(a, b, __float_as_uint(fmaf(__uint_as_float(d), 0x1p-5f, __uint_as_float(c))));
}

// A part in the scratch: O of every head, then m and l.
template <int HD, int G>
EE_DEV float* part(const DecodeParams& p, int slot) {
  return static_cast<float*>(p.scratch) + (size_t)slot * G * (HD + 2);
}

template <int HD, int G>
__global__ void __launch_bounds__(kThreads, Layout<HD, G>::kCtas)
    k_quantized_attention(const DecodeParams p, const __grid_constant__ CUtensorMap map, const float c, const int least,
                          const bool whole) {
  using Lay = Layout<HD, G>;
  constexpr int N = Lay::N, NS = Lay::NS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<HD, G> sh;
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, me = blockIdx.x;
  uint8_t *qs = ring + Lay::oQ, *xs = ring + Lay::oX, *es = ring + Lay::oE;
  grid_dep_launch();
  // Tiles and shares count on; after a wait that gave up the loops go on without waiting:
  // every thread still meets the barriers that count threads.
  bool ok = true;

  // The loads begin before anything else is ready: their warp makes the barriers, and
  // does not wait for the others.
  if (warp == 4) {
    sh.shares.init(7);
    if (lane == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(&sh.full[i], 33);  // the copies' bytes; 32 lanes' exponents
        mbar_init(&sh.empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.s_full[i], 1);
        mbar_init(&sh.q_ready[i], 64);
        mbar_init(&sh.q_free[i], 5);  // the products with it, and four warps that have its scales
      }
      mbar_init(&sh.x_ready, 128);
      mbar_init(&sh.o_done, 1);
      mbar_init(&sh.drained, 1);
      fence_mbar_init();
    }
    __syncwarp();
    asm volatile("bar.arrive 2, 256;" ::: "memory");
  }
  if (warp != 4) {
    if (warp == 5) {
      tmem_alloc(&sh.tmem, 4 * N);
      tc_fence_before();
    }
    asm volatile("bar.sync 2, 256;" ::: "memory");
    tc_fence_after();
  }
  const uint32_t tmem = warp == 4 ? 0 : sh.tmem;
  auto s_col = [&](int t) { return tmem + (t & 1) * N; };
  auto o_col = [&](int r) { return tmem + 2 * N + (r & 1) * N; };

  if (warp == 4) {
    DecodePlan plan;
    plan.init(p, gridDim.x, least, whole, me);
    const uint64_t once = l2_evict_first_policy();
    int t = 0, n = 0, at = plan.begin;
    auto next = [&]() {
      const Share w = plan.at(&at, me);
      ok = ok && sh.shares.put(n++, w, p.c.err);
      return w;
    };
    Share u = next();
    while (u.s >= 0 && ok) {
      const Share then = next();  // known before this one's last tile is issued
      if (!ok) break;
      const int32_t* table = p.c.table + (int64_t)u.s * p.c.table_stride + u.first;
      int ids = 0;
      for (int j = 0; j < u.blocks && ok; j += 8, ++t) {
        // block ids come 32 at a time
        if ((j & 31) == 0) ids = j + lane < u.blocks ? table[j + lane] : 0;
        const int here = min(8, u.blocks - j), st = t % NS;
        int id = __shfl_sync(0xffffffffu, ids, (j & 31) + (lane & 7)), eid = __shfl_sync(0xffffffffu, ids, (j & 31) + (lane >> 2));
        if (id < 0 || id >= p.c.n_blocks) {
          if (lane < here) report(p.c.err, EE_DERR_BLOCK);
          id = 0;
        }
        if (eid < 0 || eid >= p.c.n_blocks) eid = 0;
        if (t >= NS) ok = warp_wait(&sh.empty[st], (t / NS - 1) & 1, p.c.err, DERR_EMPTY_WAIT);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], (uint32_t)here * Lay::kBlock);
        __syncwarp();
        if (lane < here)
          tma_stream_5d(smem_addr(ring + st * Lay::kTile + lane * Lay::kBlock), &map, 0, 0, 0, 0, id * p.c.n_kv_heads + u.g,
                        &sh.full[st], once);
        if ((lane >> 2) < here)
          copy8(smem_addr(es + st * 256 + lane * 8), p.exponents + ((int64_t)eid * p.c.n_kv_heads + u.g) * 32 + (lane & 3) * 8);
        copies_arrive(&sh.full[st]);
      }
      u = then;
    }
    // empty sequences
    for (int s = me; s < p.batch; s += gridDim.x)
      if (__shfl_sync(0xffffffffu, s < 32 ? plan.tokens[0] : plan.tokens[1], s & 31) == 0)
        for (int i = lane * 8; i < p.n_heads * HD; i += 256)
          *reinterpret_cast<uint4*>(p.o + s * p.o_stride + i) = make_uint4(0, 0, 0, 0);
    // Copies land before the CTA ends, whichever warp gave up (where none did, they have).
    for (int i = max(0, t - NS); i < t; ++i)
      mbar_wait_bounded(&sh.full[i % NS], (uint32_t)(i / NS) & 1, p.c.err, DERR_DRAIN_WAIT);
  } else if (warp == 5) {
    constexpr uint32_t id_s = instr_desc_e4m3(N, kTokens), id_o = instr_desc_e4m3(N, HD, true, true);
    auto scores = [&](int t, int r, bool last) {  // of a tile of share r
      tc_fence_after();
      const uint64_t k = smem_desc_rows<HD>(smem_addr(ring + t % NS * Lay::kTile), Lay::kRows8),
                     q = smem_desc_rows<HD>(smem_addr(qs + (r & 1) * Lay::kQ), 8 * HD);
#pragma unroll
      for (int kk = 0; kk < HD / 32; ++kk) mma_f8(s_col(t), k + kk * 2, q + kk * 2, id_s, kk > 0);
      mma_commit(&sh.s_full[t & 1]);
      if (last) mma_commit(&sh.q_free[r & 1]);
    };
    int t = 0;
    bool out = false;  // tile t's scores
    Share u;
    ok = sh.shares.get(0, &u, p.c.err);
    for (int r = 0; ok && u.s >= 0; ++r) {
      Share then;
      if (!(ok = sh.shares.get(r + 1, &then, p.c.err))) break;
      const int tiles = (u.blocks + 7) >> 3;
      if (lane == 0) {
        for (int j = 0; j < tiles && ok; ++j, ++t) {
          auto landed = [&](int t, int r) {
            return mbar_wait_bounded(&sh.q_ready[r & 1], (r >> 1) & 1, p.c.err, DERR_FULL_WAIT) &&
                   mbar_wait_bounded(&sh.full[t % NS], (t / NS) & 1, p.c.err, DERR_FULL_WAIT);
          };
          if (!out) {
            if (!(ok = landed(t, r))) break;
            scores(t, r, j + 1 == tiles);
          }
          // The next tile's scores as soon as it is there, of this share or of the next; but the
          // product with X does not wait for them: a tile of the ring is free behind it.
          const int rn = j + 1 < tiles ? r : r + 1;
          const bool more = j + 1 < tiles || then.s >= 0, last = j + 1 < tiles ? j + 2 == tiles : then.blocks <= 8;
          out = false;
          Patience patience;
          while (!mbar_test(&sh.x_ready, t & 1)) {
            if (more && !out && mbar_test(&sh.q_ready[rn & 1], (rn >> 1) & 1) && mbar_test(&sh.full[(t + 1) % NS], ((t + 1) / NS) & 1)) {
              scores(t + 1, rn, last);
              out = true;
            }
            if (patience.over(p.c.err, DERR_FULL_WAIT)) {
              ok = false;
              break;
            }
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t v = smem_desc_rows<HD>(smem_addr(ring + t % NS * Lay::kTile) + 8 * HD, Lay::kRows8),
                         x = smem_desc_rows<32>(smem_addr(xs), 256);
#pragma unroll
          for (int kk = 0; kk < kTokens / 32; ++kk)
            mma_f8(o_col(r), v + kk * (4 * Lay::kRows8 >> 4), x + kk * (1024 >> 4), id_o, j > 0 || kk > 0);
          mma_commit(&sh.empty[t % NS]);
          mma_commit(&sh.o_done);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      t = __shfl_sync(0xffffffffu, t, 0);
      u = then;
    }
    if (lane == 0) {  // and so are the products, before tensor memory is given back
      mma_commit(&sh.drained);
      mbar_wait_bounded(&sh.drained, 0, p.c.err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else if (warp >= 6) {
    constexpr int kHeads = (G + 1) / 2, kPer = HD / 32;
    Share u;
    for (int r = 0; ok && sh.shares.get(r, &u, p.c.err) && u.s >= 0; ++r) {
      const uint16_t* q = p.q + u.s * p.q_stride + (int64_t)u.g * G * HD;
      float x[kHeads][kPer];
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = 2 * i + warp - 6;
        // neighbouring dims in a lane, whose codes are stored together
        uint32_t w[kPer / 2] = {};
        if (h < G) {
          if constexpr (HD == 128) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(q + h * HD + lane * 4);
          else w[0] = *reinterpret_cast<const uint32_t*>(q + h * HD + lane * 2);
        }
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
          x[i][2 * e] = f.x;
          x[i][2 * e + 1] = f.y;
        }
      }
      if (r >= 2) ok = warp_wait(&sh.q_free[r & 1], (r / 2 - 1) & 1, p.c.err, DERR_EMPTY_WAIT);
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = 2 * i + warp - 6;
        float big = 0.0f;
        bool fine = true;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          big = fmaxf(big, fabsf(x[i][e]));
          fine = fine && fabsf(x[i][e]) < INFINITY;
        }
        big = warp_max(big);
        fine = __all_sync(0xffffffffu, fine);
        // 2^k with 2^7 <= big 2^k < 2^8; an fp16 value's exponent is -24 or more
        const int k = fine ? min(31, 134 - (int)(__float_as_uint(big) >> 23)) : 0;
        const float up = fine ? pow2(k) : __uint_as_float(0x7fffffffu);
        if (h < G) {
          if (lane == 0) sh.unscale[r & 1][h] = c * pow2(-k);
#pragma unroll
          for (int e = 0; e < kPer; e += 2) {
            uint32_t a[3];
            parts(x[i][e] * up, x[i][e + 1] * up, a);
            const int d = lane * kPer + e;
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              const int n = part * G + h;
              *reinterpret_cast<uint16_t*>(qs + (r & 1) * Lay::kQ + (n >> 3) * 8 * HD + row_chunk<HD>(n & 7, d >> 4) + (d & 15)) =
                  (uint16_t)a[part];
            }
          }
        }
      }
      fence_proxy_async();
      mbar_arrive(&sh.q_ready[r & 1]);
    }
  } else {
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    // M = 64: rows 16 w .. 16 w + 15 in the first lanes of warp w's part of tensor memory
    const int dim = HD == 128 ? tid : warp * 16 + (lane & 15);
    const bool has_dim = HD == 128 || lane < 16;
    int t = 0;
    Share u;
    for (int r = 0;; ++r) {
      // the four warps go on together or not at all
      int go = sh.shares.get(r, &u, p.c.err) && u.s >= 0;
      asm volatile(
          "{ .reg .pred p, q; setp.ne.s32 p, %0, 0; barrier.cta.red.and.pred q, 1, 128, p; selp.s32 %0, 1, 0, q; }"
          : "+r"(go)
          :
          : "memory");
      if (!go) break;
      const int tiles = (u.blocks + 7) >> 3;
      if (ok) ok = warp_wait(&sh.q_ready[r & 1], (r >> 1) & 1, p.c.err, DERR_FULL_WAIT);
      float unscale[G], m[G], l[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        unscale[h] = sh.unscale[r & 1][h];
        m[h] = -INFINITY;
        l[h] = 0.0f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_free[r & 1]);
#pragma unroll 1
      for (int j = 0; j < tiles; ++j, ++t) {
        if (ok) ok = warp_wait(&sh.s_full[t & 1], (t >> 1) & 1, p.c.err, DERR_FULL_WAIT);
        // K's scores are made, so the tile has landed; a wait of its own orders its exponents
        if (ok) ok = warp_wait(&sh.full[t % NS], (t / NS) & 1, p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        uint32_t v[N];
        if constexpr (N == 32) tmem_ld32(s_col(t) + lane_base, v);
        else tmem_ld16(s_col(t) + lane_base, v);
        const int8_t* e8 = reinterpret_cast<const int8_t*>(es) + t % NS * 256 + (tid >> 4) * 32 + (tid & 15);
        const int ek = e8[0], ev = e8[16];
        tmem_wait_ld();
        tmem_pin<N>(v);
        const int left = u.have - j * kTokens;  // tokens from this tile on
        const bool live = tid < left;
        const float up = pow2(ek), evf = (float)ev, down = live ? pow2(-ev) : 0.0f;
        float w[G], a[G];
        int grow = 0;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          w[h] = live ? fmaf(joined(v[h], v[G + h], v[2 * G + h]) * unscale[h], up, evf) : -INFINITY;
          grow |= w[h] - m[h] > kLag;
          a[h] = 1.0f;
        }
        asm volatile(
            "{ .reg .pred p, q; setp.ne.s32 p, %0, 0; barrier.cta.red.or.pred q, 1, 128, p; selp.s32 %0, 1, 0, q; }"
            : "+r"(grow)
            :
            : "memory");
        if (grow) {  // the first tile, and rarely later
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float x = warp_max(w[h]);
            if (lane == 0) sh.red[warp][h] = x;
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float mn = fmaxf(fmaxf(fmaxf(sh.red[0][h], sh.red[1][h]), fmaxf(sh.red[2][h], sh.red[3][h])), m[h]);
            a[h] = m[h] == mn ? 1.0f : ex2(m[h] - mn);
            m[h] = mn;
            l[h] *= a[h];
          }
        }
        uint32_t x8[8] = {};  // the token's row of X: bytes part * G + h
#pragma unroll
        for (int h = 0; h < G; h += 2) {
          float x[2] = {0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < (G == 1 ? 1 : 2); ++i) {
            x[i] = ex2(w[h + i] - (m[h + i] == -INFINITY ? 0.0f : m[h + i]) + kLift);
            l[h + i] = live ? fmaf(x[i], down, l[h + i]) : l[h + i];
          }
          uint32_t cs[4];
          parts(x[0], x[1], cs);
#pragma unroll
          for (int part = 0; part < 4; ++part) {
            const int n = part * G + h;
            x8[n >> 2] |= (G == 1 ? cs[part] & 0xffu : cs[part]) << (8 * (n & 3));
          }
        }
        // the product before has read X and is in O
        if (t > 0 && ok) ok = warp_wait(&sh.o_done, (t - 1) & 1, p.c.err, DERR_FULL_WAIT);
        *reinterpret_cast<uint4*>(xs + (tid >> 3) * 256 + row_chunk<32>(tid & 7, 0)) = make_uint4(x8[0], x8[1], x8[2], x8[3]);
        if constexpr (N == 32)
          *reinterpret_cast<uint4*>(xs + (tid >> 3) * 256 + row_chunk<32>(tid & 7, 1)) = make_uint4(x8[4], x8[5], x8[6], x8[7]);
        if (left < kTokens) {
          // slots behind the last token hold anything: their V becomes zero
          uint8_t* tile = ring + t % NS * Lay::kTile + 8 * HD;
          for (int i = left * (HD / 16) + tid; i < kTokens * (HD / 16); i += 128) {
            const int row = i / (HD / 16);
            *reinterpret_cast<uint4*>(tile + (row >> 3) * Lay::kRows8 + (row & 7) * HD + (i % (HD / 16)) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        if (grow && j > 0) {
          tc_fence_after();
          uint32_t o[N];
          if constexpr (N == 32) tmem_ld32(o_col(r) + lane_base, o);
          else tmem_ld16(o_col(r) + lane_base, o);
          tmem_wait_ld();
          tmem_pin<N>(o);
#pragma unroll
          for (int i = 0; i < 4 * G; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a[i % G]);
          tmem_st16(o_col(r) + lane_base, o);
          if constexpr (N == 32) tmem_st16(o_col(r) + 16 + lane_base, o + 16);
          tmem_wait_st();
        }
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&sh.x_ready);
      }
      // the share's end: l of all warps, O of this thread's dim
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float x = warp_sum(l[h]);
        if (lane == 0) sh.sum[warp][h] = x;
      }
      if (ok) ok = warp_wait(&sh.o_done, (t - 1) & 1, p.c.err, DERR_FULL_WAIT);
      tc_fence_after();
      uint32_t o[N];
      if constexpr (N == 32) tmem_ld32(o_col(r) + lane_base, o);
      else tmem_ld16(o_col(r) + lane_base, o);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      tmem_wait_ld();
      tmem_pin<N>(o);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float sum = (sh.sum[0][h] + sh.sum[1][h]) + (sh.sum[2][h] + sh.sum[3][h]);
        const float y = joined(o[h], o[G + h], o[2 * G + h], o[3 * G + h]);
        if (u.slot < 0) {
          if (has_dim && ok) p.o[u.s * p.o_stride + (u.g * G + h) * HD + dim] = float_to_half_bits(within_half(__fdividef(y, sum)));
        } else {
          float* to = part<HD, G>(p, u.slot);
          if (has_dim) to[h * HD + dim] = y;
          if (tid == h) {
            to[G * HD + h] = m[h];
            to[G * HD + G + h] = sum;
          }
        }
      }
      // sum is read before the next share's is written: its first tile's barrier is between
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_free(tmem, 4 * N);
  }
  if (!ok) __nanosleep(1000000);  // what this CTA no longer waited for may be on its way
}

// Adds the parts of pairs that several CTAs had a share of.
template <int HD, int G, int J>
__global__ void __launch_bounds__(kJoinThreads) k_join(const DecodeParams p, const int pieces, const int least) {
  using Sum = Join<HD, J>;
  constexpr int P = Sum::P, U = Sum::kAtOnce, kStripes = Sum::kStripes;
  __shared__ typename Sum::Stripes stripes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x / (p.n_heads / J), first = (blockIdx.x - s * (p.n_heads / J)) * J;  // its heads
  const int g = first / G, h = first % G + warp % J;
  DecodePlan plan;
  plan.init(p, pieces, least, false, 0);
  const int nb = (__shfl_sync(0xffffffffu, s < 32 ? plan.tokens[0] : plan.tokens[1], s & 31) + 15) >> 4;
  const int from = __shfl_sync(0xffffffffu, s < 32 ? plan.base[0] : plan.base[1], s & 31) * plan.hkv +
                   g * __shfl_sync(0xffffffffu, s < 32 ? plan.size[0] : plan.size[1], s & 31);
  const DecodePieces::Parts parts = plan.parts(from, nb);
  const int n = parts.count;
  grid_dep_wait();
  if (n < 2) return;
  Sum sum;
  for (int k0 = warp / J; k0 < n; k0 += kStripes * U) {
    float mk[U], lk[U], x[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + kStripes * u;
      const float* y = part<HD, G>(p, parts.slot(k));
      mk[u] = -INFINITY;
      lk[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < P; ++i) x[u][i] = 0.0f;
      if (k < n) {
        mk[u] = y[G * HD + h];
        lk[u] = y[G * HD + G + h];
        if constexpr (P == 4 && G > 1) *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(y + h * HD + lane * P);
        else
#pragma unroll
          for (int i = 0; i < P; i += 2)
            *reinterpret_cast<float2*>(x[u] + i) = *reinterpret_cast<const float2*>(y + h * HD + lane * P + i);
      }
    }
    sum.add(mk, lk, x);
  }
  sum.finish(stripes, p.o + s * p.o_stride + first * HD);
}

template <int HD, int G>
cudaError_t launch_t(const DecodeParams& p, cudaStream_t st) {
  using Lay = Layout<HD, G>;
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_quantized_attention<HD, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  CUtensorMap map;
  // a block of a kv head, as groups of 8 tokens: [group][K, V][8][HD]
  const uint64_t d[5] = {(uint64_t)HD, 8, 2, 2, (uint64_t)p.c.n_blocks * p.c.n_kv_heads},
                 s[4] = {(uint64_t)HD, (uint64_t)HD * 16, (uint64_t)HD * 8, (uint64_t)HD * 32};
  const uint32_t b[5] = {(uint32_t)HD, 8, 2, 2, 1};
  if (!encode_tensor_map_bytes(&map, 5, p.codes, d, s, b)) return cudaErrorInvalidValue;
  const int64_t most = (int64_t)p.batch * p.c.n_kv_heads * (DecodePlan::kStart + (p.c.max_ctx + 15) / 16);
  const int least = 8;
  const bool whole = p.c.max_ctx <= kTokens;
  const int pieces = (int)std::min<int64_t>(std::min(Lay::kCtas * sms, kMaxCtas), (most + least - 1) / least);
  k_quantized_attention<HD, G><<<pieces, kThreads, Lay::kSmem, st>>>(p, map, 1.44269504f / sqrtf((float)HD), least, whole);
  e = cudaGetLastError();
  if (e != cudaSuccess || whole) return e;
  return join_by_rows<G>(p.batch * p.n_heads, sms, [&](auto J) {
    return launch_join(k_join<HD, G, J.value>, p.batch * (p.n_heads / J.value), sms, Lay::kSmem, st, p, pieces, least);
  });
}

}  // namespace

cudaError_t launch_quantized_attention(const DecodeParams& p, cudaStream_t st) {
  const int G = p.n_heads / p.c.n_kv_heads, hd = p.c.head_dim;
#define EE_DECODE_CASE(HD_, G_) \
  if (hd == HD_ && G == G_) return launch_t<HD_, G_>(p, st);
  EE_DECODE_CASE(64, 1)
  EE_DECODE_CASE(64, 2)
  EE_DECODE_CASE(64, 4)
  EE_DECODE_CASE(64, 8)
  EE_DECODE_CASE(128, 1)
  EE_DECODE_CASE(128, 2)
  EE_DECODE_CASE(128, 4)
  EE_DECODE_CASE(128, 8)
#undef EE_DECODE_CASE
  return cudaErrorInvalidValue;
}

size_t quantized_attention_scratch(int32_t, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t) {
  return (size_t)2 * kMaxCtas * (n_heads / n_kv_heads) * (head_dim + 2) * 4;
}

}  // namespace ee
