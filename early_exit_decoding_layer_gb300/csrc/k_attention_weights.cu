// Decode attention over the paged cache that also adds what each token weighs, on
// the tensor cores.
//
// One new token per sequence: K and V are read once for the G query heads of a kv
// head, 2 G products per element, so the bytes are the bound -- if the arithmetic
// keeps out of the way.  On the CUDA cores (a token per lane, fp32 fma) it did not:
// 1100 instructions per 16-slot block and warp held 32 sequences of up to 2176
// tokens at 45 us, where the bytes take 23.  So both products run as MMAs with
// the cache as the big operand:
//   S = K_tile Q^T    128 tokens x 16 columns
//   O^T = V_tile^T P  head dims x 16 columns, K = 128 tokens
// fp32 queries and probabilities go in as fp16 pairs, x = hi + lo, columns h and
// 8 + h: 22 bits, which keeps the fp32 result.  A query head is scaled by a power
// of two to a largest value near 2^10, and probabilities by 2^7, so that neither
// part falls below fp16's range.  Each tile's O is a product of its own, added to
// fp32 registers: the tensor core cuts its accumulator after every step, which
// over 16384 tokens would show.
//
// A cluster of C CTAs serves one (sequence, kv head) after another, each CTA a share
// of its 16-slot blocks, in tiles of eight:
//   warps 0-3  a thread per token: scores, a running maximum that may lag by 2^8 (so
//              that rescaling is rare), probabilities into shared memory;
//              then a thread per head dim adds O
//   warps 4-7  the next unit's Q; the join of the last unit and its tokens' weights
//   warp 8     K and V tiles by TMA into a ring, over the ends of the units
//   warp 9     (one thread) the MMAs, S a tile ahead of O
// The scores of a share stay in shared memory.  At the end of a unit every CTA pushes
// its m and l to all ranks, and its O to the rank that writes that part of the
// output (st.async, counted on the receiver's barrier: neither fence nor answer).
// Receivers add in rank order, and each turns its own scores into weights.  One
// launch, no scratch, K and V read once.
//
// A box of the TMA is a whole block, [2 groups][halves][8 rows][128 bytes]: with boxes of
// one half, as they would lie in a plain tile, they came one in 78 cycles and a tile
// took 1.3 us at best, now 1.0.  Units that follow each other in a CTA without a
// pause, against a CTA per unit with two on an SM: 39 -> 35 us for 32 sequences of 257
// to 2176 tokens, 210 -> 197 for 32 of 8192 (32/8 heads, hd 128).
//
// Bound: bytes.  32 sequences of 8192 tokens, 32/8 heads, hd 128: 5.5 TB/s (0.82 of
// the measured copy rate); 257 to 2176 tokens: 4.5 TB/s, where 152 SMs share 256 units
// unevenly and 5.5 us of launch, first loads and last join show; one of 2113: 8.3 us.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "ee_cache_ops.cuh"
#include "ee_tcgen05.cuh"

namespace cg = cooperative_groups;

namespace ee {
namespace {

constexpr int kThreads = 320;
constexpr int kTokens = 128;  // per tile, eight blocks
constexpr int kMaxCluster = 12;
constexpr float kLift = 7.0f;  // probabilities are 2^kLift times their value

struct Maps {
  CUtensorMap k, v;
};

template <int HD>
struct Layout {
  static constexpr int H = HD / 64;                     // 64-column halves
  static constexpr uint32_t kTile = kTokens * HD * 2;   // K or V of one tile
  static constexpr uint32_t kGroup = H * 1024;          // 8 tokens of it: [half][8][64]
  static constexpr int kMost = 10;                      // ring tiles at most
  static constexpr uint32_t kQ = H * 2048, kP = 4096;   // 16 rows of 128 bytes for every 64 columns
};

// Shared memory behind the ring of `ns` tiles: Q and P twice, all ranks' O of this
// rank's share of the outputs three times, the scores of a share of the tokens
// (`cap`) once or twice, its block ids.
template <int HD, int G>
struct Parts {
  using Lay = Layout<HD>;
  static constexpr int kOuts = G * HD + 16;  // C * ceil(G * HD / C) at most
  static constexpr int kQ = 0, kP = kQ + 2 * Lay::kQ, kO = kP + 2 * Lay::kP, kScores = kO + 3 * kOuts * 4;
  static size_t bytes(int cap, int buffers) { return kScores + (size_t)cap * G * 4 * buffers + cap / 16 * 4; }
};

template <int HD, int G>
struct Shared {
  uint64_t full[Layout<HD>::kMost], empty[Layout<HD>::kMost], s_full[2], p_ready[2], o_full[2];
  uint64_t q_ready[2], part_full[2], part_free[2];  // by unit & 1
  uint64_t drained;                                 // every MMA issued is over
  uint64_t joined[3];                               // every rank's part of a unit is there; by unit % 3
  uint32_t tmem;
  int order[EE_MAX_BATCH], tokens[EE_MAX_BATCH];  // sequences by falling length
  float unscale[2][8], red[4][8];
  float m[3][kMaxCluster][G], l[3][kMaxCluster][4][G];  // of every rank, l by warp
  float sum[kMaxCluster][G];
  float f[kMaxCluster][G];                       // what a rank's O counts in the whole
  float M[G], inv[G];                            // of the whole sequence
};

// A place in the ring.
struct Slot {
  int at = 0;
  uint32_t phase = 0;
  EE_DEV void next(int ns) {
    if (++at == ns) {
      at = 0;
      phase ^= 1;
    }
  }
};

// Sequences and their tokens by falling position (equal ones by index); a whole warp.
EE_DEV void sort_sequences(const DecodeWeightsParams& p, int* order, int* tokens) {
  static_assert(EE_MAX_BATCH <= 64, "two sequences per lane");
  const int lane = threadIdx.x & 31;
  const int a = lane < p.batch ? p.pos[lane] : INT_MIN, b = lane + 32 < p.batch ? p.pos[lane + 32] : INT_MIN;
  int ra = 0, rb = 0;  // how many come before
#pragma unroll 4
  for (int k = 0; k < min(p.batch, 32); ++k) {
    const int x = __shfl_sync(0xffffffffu, a, k), y = __shfl_sync(0xffffffffu, b, k);
    ra += (x > a || (x == a && k < lane)) + (y > a);
    rb += (x >= b) + (y > b || (y == b && k < lane));
  }
  auto put = [&](int s, int rank, int at) {
    if (s >= p.batch) return;
    order[rank] = s;
    tokens[rank] = checked_length(at == INT32_MAX ? at : at + 1, p.c.max_ctx, p.c.err);
  };
  put(lane, ra, a);
  put(lane + 32, rb, b);
}

// What a CTA does for one (sequence, kv head).
struct Work {
  int s, g, blocks, first, tiles, have;  // s = -1: no more; its blocks from `first` on, its tokens
};

// Writes to the same place in the CTA of that rank, counted in bytes on its barrier.
EE_DEV void push(float* to, float value, uint64_t* bar, int rank) {
  asm volatile(
      "{ .reg .b32 a, b; mapa.shared::cluster.u32 a, %0, %2; mapa.shared::cluster.u32 b, %1, %2; "
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [a], %3, [b]; }" ::"r"(smem_addr(to)),
      "r"(smem_addr(bar)), "r"(rank), "r"(__float_as_uint(value))
      : "memory");
}

// hi + lo of a value that went in as two fp16 parts.  Where hi is not finite, lo is no
// part of it (0 times infinity).
EE_DEV float whole(uint32_t hi, uint32_t lo) {
  return (hi & 0x7f800000u) == 0x7f800000u ? __uint_as_float(hi) : __uint_as_float(hi) + __uint_as_float(lo);
}

template <int HD, int G>
__global__ void __launch_bounds__(kThreads, 1)
    k_attention_weights(const DecodeWeightsParams p, const __grid_constant__ Maps maps, const float c, const int ns,
                        const int buffers) {
  using Lay = Layout<HD>;
  using Part = Parts<HD, G>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<HD, G> sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = ((p.c.max_ctx + 15) / 16 + C - 1) / C * 16;  // tokens of a CTA at most
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* parts = ring + ns * Lay::kTile;
  uint8_t* qs = parts + Part::kQ;
  uint8_t* ps = parts + Part::kP;
  float* outs = reinterpret_cast<float*>(parts + Part::kO);  // [3][kOuts]: [rank][share]
  float* scores = reinterpret_cast<float*>(parts + Part::kScores);  // [buffers][G][cap], in log2 units
  int* ids = reinterpret_cast<int*>(scores + (size_t)buffers * G * cap);  // [cap / 16], -1 where out of range

  // A cluster's r-th unit: long sequences first, every second round in the opposite order.
  const int nc = gridDim.x / C, me = blockIdx.x / C;
  auto work = [&](int r) {
    const int unit = r * nc + ((r & 1) ? nc - 1 - me : me);
    Work w;
    w.s = -1;
    if (unit >= p.batch * p.c.n_kv_heads) return w;
    const int at = unit / p.c.n_kv_heads;
    w.s = sh.order[at];
    w.g = unit - at * p.c.n_kv_heads;
    const int n = sh.tokens[at], nb = (n + 15) >> 4, each = (nb + C - 1) / C;
    w.first = min(nb, rank * each);
    w.blocks = min(nb, w.first + each) - w.first;
    w.tiles = (w.blocks + 7) >> 3;
    w.have = max(0, min(n - w.first * 16, w.blocks * 16));
    return w;
  };

  if (tid < Lay::kMost) {
    mbar_init(&sh.full[tid], 1);
    mbar_init(&sh.empty[tid], 1);
    fence_mbar_init();
  } else if (tid >= 32 && tid < 34) {  // by the two buffers
    const int i = tid - 32;
    mbar_init(&sh.s_full[i], 1);
    mbar_init(&sh.p_ready[i], 128);
    mbar_init(&sh.o_full[i], 1);
    mbar_init(&sh.q_ready[i], 128);
    mbar_init(&sh.part_full[i], 129);  // the softmax warps, and the MMA thread past q_ready
    mbar_init(&sh.part_free[i], 128);
    fence_mbar_init();
  } else if (tid >= 64 && tid < 67) {
    mbar_init(&sh.joined[tid - 64], 1);
    if (tid == 64) mbar_init(&sh.drained, 1);
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&sh.tmem, 64);
  if (warp == 8) sort_sequences(p, sh.order, sh.tokens);
  // rows of Q and P without a head are zero
  for (int i = tid; i < (Part::kO - Part::kQ) / 16; i += kThreads) reinterpret_cast<uint4*>(qs)[i] = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // First phase of the cluster's barrier: the barriers of all ranks are in place;
  // waited for before the first push.  Second phase: this thread pushes no more;
  // waited for before the end, so that no CTA is gone while another could still
  // write to it.
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  auto cluster_ready = [] { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); };
  auto cluster_done = [] { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); };
  const int share = (G * HD + C - 1) / C;  // outputs per rank
  const uint32_t tmem = sh.tmem;
  // Ring items, and the tiles that the S, P and O buffers alternate with, count on
  // over the units.  After a wait that gave up the loops go on without waiting:
  // every thread still meets the barriers that count threads.
  bool ok = true;

  if (warp == 8) {
    // ring item 2 t is K of tile t, item 2 t + 1 its V
    Slot slot;
    int issued = 0;
    // block ids come 32 at a time, a group ahead of their use: one read per tile
    // in its turn took longer (1.4 us) than the tile
    auto ids32 = [&](const Work& w, int q) {
      const int b = 32 * q + lane;
      return w.s >= 0 && b < w.blocks ? p.c.table[(int64_t)w.s * p.c.table_stride + w.first + b] : 0;
    };
    Work w = work(0);
    int now = ids32(w, 0);
    for (int r = 0; w.s >= 0 && ok; ++r) {
      const Work then = work(r + 1);
      const int first = ids32(then, 0);
      int ahead = ids32(w, 1);
      for (int j = 0; j < w.tiles && ok; ++j) {
        if (j > 0 && j % 4 == 0) {
          now = ahead;
          ahead = ids32(w, j / 4 + 1);
        }
        const int here = min(8, w.blocks - 8 * j);
        int id = __shfl_sync(0xffffffffu, now, j % 4 * 8 + (lane & 7));
        if (id < 0 || id >= p.c.n_blocks) {
          report(p.c.err, EE_DERR_BLOCK);
          id = 0;
        }
        for (int kv = 0; kv < 2; ++kv, ++issued, slot.next(ns)) {
          if (issued >= ns) ok = warp_wait(&sh.empty[slot.at], slot.phase ^ 1, p.c.err, DERR_EMPTY_WAIT);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot.at], (uint32_t)here * 16 * HD * 2);
          __syncwarp();
          if (lane < here)
            tma_load_4d(smem_addr(ring + slot.at * Lay::kTile + lane * 2 * Lay::kGroup), kv ? &maps.v : &maps.k, 0, 0, 0,
                        (id * p.c.n_kv_heads + w.g) * 2, &sh.full[slot.at]);
        }
      }
      w = then;
      now = first;
    }
    // Copies land before the CTA ends, whichever warp gave up (where none did, they have).
    for (int i = max(0, issued - ns); i < issued; ++i)
      mbar_wait_bounded(&sh.full[i % ns], (uint32_t)(i / ns) & 1, p.c.err, DERR_DRAIN_WAIT);
    __syncwarp();
    cluster_ready();
    cluster_done();
  } else if (warp == 9) {
    if (lane == 0) {
      constexpr uint32_t id_s = instr_desc(0, 16, kTokens), id_o = instr_desc(0, 16, HD, false, true);
      Slot slot;  // K of the next tile whose scores go out
      int t = 0;  // tile
      auto landed = [&](const Slot& x) {
        const bool r = mbar_wait_bounded(&sh.full[x.at], x.phase, p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        return r;
      };
      Work w = work(0);
      for (int r = 0; w.s >= 0 && ok; w = work(++r)) {
        const uint64_t qd = smem_desc_sw128(smem_addr(qs) + (r & 1) * Lay::kQ);
        if (!(ok = mbar_wait_bounded(&sh.q_ready[r & 1], (r >> 1) & 1, p.c.err, DERR_FULL_WAIT))) break;
        // Where this CTA has no tile nobody waits for this thread's products: without this
        // arrival Q of unit r + 2 could be placed before it has seen that of unit r.
        mbar_arrive(&sh.part_full[r & 1]);
        Slot vs[2];  // V of tile t, by t & 1
        auto issue_scores = [&](int t) {
          if (!landed(slot)) return false;
          const uint64_t k = smem_desc_sw128(smem_addr(ring) + slot.at * Lay::kTile, Lay::kGroup);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_f16(tmem + (t & 1) * 16, k + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                    qd + (((kk >> 2) * 2048 + (kk & 3) * 32) >> 4), id_s, kk > 0);
          mma_commit(&sh.s_full[t & 1]);
          slot.next(ns);
          if (t & 1) vs[1] = slot;
          else vs[0] = slot;
          slot.next(ns);
          return true;
        };
        const int end = t + w.tiles;
        if (t < end) ok = issue_scores(t);
#pragma unroll 1
        for (; t < end && ok; ++t) {
          if (t + 1 < end && !(ok = issue_scores(t + 1))) break;
          const Slot v_at = t & 1 ? vs[1] : vs[0];
          if (!(ok = mbar_wait_bounded(&sh.p_ready[t & 1], (t >> 1) & 1, p.c.err, DERR_FULL_WAIT) && landed(v_at))) break;
          const uint64_t v = smem_desc_sw128_mn(smem_addr(ring) + v_at.at * Lay::kTile, 1024, Lay::kGroup);
          const uint64_t pd = smem_desc_sw128(smem_addr(ps) + (t & 1) * Lay::kP);
#pragma unroll
          for (int kk = 0; kk < kTokens / 16; ++kk)
            mma_f16(tmem + 32 + (t & 1) * 16, v + kk * (2 * Lay::kGroup >> 4), pd + (((kk >> 2) * 2048 + (kk & 3) * 32) >> 4), id_o,
                    kk > 0);
          mma_commit(&sh.o_full[t & 1]);
        }
      }
      // and so are the products, before tensor memory is given back
      mma_commit(&sh.drained);
      mbar_wait_bounded(&sh.drained, 0, p.c.err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
    cluster_ready();
    cluster_done();
  } else if (warp < 4) {
    Slot slot;  // K of the next tile
    int t = 0, buf3 = 0;
    uint32_t phase3 = 0;  // of unit r: r % 3, r / 3 & 1
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    Work u = work(0);
    for (int r = 0; u.s >= 0; u = work(++r)) {
      const int buf = r & 1, have = u.have;
      float* sc = scores + (buffers == 2 ? (size_t)buf * G * cap : 0);
      // this unit's scores: the join of the one whose buffer they take is done
      const int joined = r - buffers;
      if (joined >= 0 && ok) ok = warp_wait(&sh.part_free[joined & 1], (joined >> 1) & 1, p.c.err, DERR_EMPTY_WAIT);
      if (ok) ok = warp_wait(&sh.q_ready[buf], (r >> 1) & 1, p.c.err, DERR_FULL_WAIT);
      float unscale[G], m[G], l[G], acc[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        unscale[h] = sh.unscale[buf][h];
        m[h] = -INFINITY;
        l[h] = 0.0f;
        acc[h] = 0.0f;
      }
      int v_before = 0;  // the ring's place of the V before
      auto add_output = [&](int t, int v_at) {
        if (ok) ok = warp_wait(&sh.o_full[t & 1], (t >> 1) & 1, p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        if (tid == 0) mbar_arrive(&sh.empty[v_at]);
        uint32_t v[16];
        tmem_ld16(tmem + 32 + (t & 1) * 16 + lane_base, v);
        tmem_wait_ld();
        tmem_pin<16>(v);
#pragma unroll
        for (int h = 0; h < G; ++h) acc[h] += whole(v[h], v[8 + h]);
      };
#pragma unroll 1
      for (int j = 0; j < u.tiles; ++j, ++t) {
        if (ok) ok = warp_wait(&sh.s_full[t & 1], (t >> 1) & 1, p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        if (tid == 0) mbar_arrive(&sh.empty[slot.at]);
        slot.next(ns);
        const Slot v_at = slot;
        slot.next(ns);
        uint32_t v[16];
        tmem_ld16(tmem + (t & 1) * 16 + lane_base, v);
        tmem_wait_ld();
        tmem_pin<16>(v);
        const int left = have - j * kTokens;  // tokens from this tile on
        const bool live = tid < left;
        float z[G], a[G];
        int grow = 0;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          z[h] = live ? whole(v[h], v[8 + h]) * unscale[h] : -INFINITY;
          grow |= z[h] - m[h] > 8.0f;
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
            const float x = warp_max(z[h]);
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
        uint8_t* pt = ps + (t & 1) * Lay::kP + (tid >> 6) * 2048 + (tid & 7) * 2;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float e = ex2(z[h] - (m[h] == -INFINITY ? 0.0f : m[h]) + kLift);
          l[h] += e;
          const __half hi = __float2half_rn(e), lo = __float2half_rn(e - __half2float(hi));
          *reinterpret_cast<__half*>(pt + sw128(h, (tid & 63) >> 3)) = hi;
          *reinterpret_cast<__half*>(pt + sw128(8 + h, (tid & 63) >> 3)) = lo;
          if (live) sc[h * cap + j * kTokens + tid] = z[h];
        }
        if (left < kTokens) {
          // slots behind the last token hold anything: their V becomes zero
          if (ok) ok = warp_wait(&sh.full[v_at.at], v_at.phase, p.c.err, DERR_FULL_WAIT);
          uint8_t* tile = ring + v_at.at * Lay::kTile;
          for (int i = left * 8 + tid; i < kTokens * 8; i += 128)
#pragma unroll
            for (int half = 0; half < Lay::H; ++half)
              *reinterpret_cast<uint4*>(tile + (i >> 6) * Lay::kGroup + half * 1024 + (i & 63) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&sh.p_ready[t & 1]);
        if (j > 0) add_output(t - 1, v_before);
        v_before = v_at.at;
#pragma unroll
        for (int h = 0; h < G; ++h) acc[h] *= a[h];
      }
      if (u.tiles > 0) add_output(t - 1, v_before);
      // (m, l, O) go to the ranks that need them.  Of three buffers each, this one is
      // free once all ranks have pushed the last unit: each began it after it had
      // joined the one two before that.
      mbar_arrive(&sh.part_full[buf]);
      if (r == 0) cluster_ready();
      if (r >= 3 && ok) {
        const int last = buf3 == 0 ? 2 : buf3 - 1;
        ok = warp_wait(&sh.joined[last], buf3 == 0 ? phase3 ^ 1 : phase3, p.c.err, DERR_EMPTY_WAIT);
      }
      // M = 64: rows 16 w .. 16 w + 15 in the first lanes of warp w's part of tensor memory
      const int dim = HD == 128 ? tid : warp * 16 + (lane & 15);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float x = warp_sum(l[h]);
        if (ok && lane < C) {
          push(&sh.l[buf3][rank][warp][h], x, &sh.joined[buf3], lane);
          if (warp == 0) push(&sh.m[buf3][rank][h], m[h], &sh.joined[buf3], lane);
        }
        if (ok && (HD == 128 || lane < 16)) {
          const int i = h * HD + dim, to = i / share;
          push(outs + buf3 * Part::kOuts + rank * share + (i - to * share), acc[h], &sh.joined[buf3], to);
        }
      }
      if (++buf3 == 3) {
        buf3 = 0;
        phase3 ^= 1;
      }
    }
    cluster_done();
    tc_fence_before();
  } else {
    // Q of the next unit ahead, then the join of this one, while the softmax warps go
    // on with the next.
    const int jt = tid - 128, jw = warp - 4;
    int buf3 = 0;
    uint32_t phase3 = 0;  // of unit r: r % 3, r / 3 & 1
    auto meet = [] { asm volatile("bar.sync 2, 128;" ::: "memory"); };
    auto first_block = [&](const Work& u) { return p.c.table + (int64_t)u.s * p.c.table_stride + u.first; };
    constexpr int kHeads = (G + 3) / 4;  // of Q per warp
    float x[kHeads][HD / 32];
    auto load_q = [&](const Work& u) {
      const float* qg = p.q + ((size_t)u.s * p.n_heads + u.g * G) * HD;
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) x[i][e] = jw + 4 * i < G ? qg[(jw + 4 * i) * HD + e * 32 + lane] * c : 0.0f;
    };
    auto place_q = [&](int buf) {
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = jw + 4 * i;
        if (h < G) {
          float big = 0.0f;
#pragma unroll
          for (int e = 0; e < HD / 32; ++e) big = fmaxf(big, fabsf(x[i][e]));
          big = warp_max(big);
          // 2^k with 2^9 <= big 2^k < 2^10; k is -119 or more, and at most 60: what is smaller
          // scores less than 2^-28 with any keys
          const int k = min(60, 136 - (int)(__float_as_uint(big) >> 23));
          const float up = __uint_as_float((uint32_t)(127 + k) << 23);
          if (lane == 0) sh.unscale[buf][h] = __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
          for (int e = 0; e < HD / 32; ++e) {
            const int d = e * 32 + lane;
            const float y = x[i][e] * up;
            const __half hi = __float2half_rn(y), lo = __float2half_rn(y - __half2float(hi));
            uint8_t* to = qs + buf * Lay::kQ + (d >> 6) * 2048 + (d & 7) * 2;
            *reinterpret_cast<__half*>(to + sw128(h, (d & 63) >> 3)) = hi;
            *reinterpret_cast<__half*>(to + sw128(8 + h, (d & 63) >> 3)) = lo;
          }
        }
      }
      fence_proxy_async();
      mbar_arrive(&sh.q_ready[buf]);
    };
    Work u = work(0);
    load_q(u);
    place_q(0);
    Work then = work(1);
    if (then.s >= 0) load_q(then);
    int first_id = jt < u.blocks ? first_block(u)[jt] : 0;
    for (int r = 0; u.s >= 0; ++r) {
      const int buf = r & 1, s = u.s, g = u.g;
      const float* sc = scores + (buffers == 2 ? (size_t)buf * G * cap : 0);
      // the products that read this buffer's last Q are done: their unit was joined
      if (then.s >= 0) place_q(buf ^ 1);
      for (int b = jt; b < u.blocks; b += 128) {
        const int id = b == jt ? first_id : first_block(u)[b];
        ids[b] = id < 0 || id >= p.c.n_blocks ? -1 : id;
      }
      // loads for the next round
      const Work later = then.s >= 0 ? work(r + 2) : then;
      if (later.s >= 0) load_q(later);
      if (then.s >= 0 && jt < then.blocks) first_id = first_block(then)[jt];
      const int first = rank * share, end = min(G * HD, first + share);  // this rank's outputs
      if (jt == 0) mbar_arrive_expect_tx(&sh.joined[buf3], (uint32_t)(C * 4 * (5 * G + max(0, end - first))));
      __syncwarp();
      if (r == 0) {
        cluster_ready();
        cluster_done();
      }
      if (ok) ok = warp_wait(&sh.part_full[buf], (r >> 1) & 1, p.c.err, DERR_FULL_WAIT);
      if (ok) ok = warp_wait(&sh.joined[buf3], phase3, p.c.err, DERR_FULL_WAIT);
      // every rank finds M and L, rank k a share of the outputs, in rank order
      if (jt < C * G) {
        static_assert(kMaxCluster * G <= 128, "a thread per rank and head");
        const int k = jt / G, h = jt % G;
        sh.sum[k][h] = (sh.l[buf3][k][0][h] + sh.l[buf3][k][1][h]) + (sh.l[buf3][k][2][h] + sh.l[buf3][k][3][h]);
      }
      meet();
      if (jt < G) {
        float mk[kMaxCluster], mm = -INFINITY, ll = 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          mk[k] = k < C ? sh.m[buf3][k][jt] : -INFINITY;
          mm = fmaxf(mm, mk[k]);
        }
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < C) {
            const float lk = sh.sum[k][jt], f = lk == 0.0f ? 0.0f : mk[k] == mm ? 1.0f : ex2(mk[k] - mm);
            sh.f[k][jt] = f;
            ll = fmaf(f, lk, ll);  // f may have gone to 0: a NaN stays
          }
        sh.M[jt] = mm == -INFINITY ? 0.0f : mm;  // scores of -inf alone: no weight, not NaN
        sh.inv[jt] = ll == 0.0f ? 0.0f : 1.0f / ll;
      }
      meet();
      const float* parts_of = outs + buf3 * Part::kOuts;
      for (int i = first + jt; i < end; i += 128) {
        const int h = i / HD;
        float a = 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < C) a = fmaf(sh.f[k][h], parts_of[k * share + i - first], a);
        p.o[((size_t)s * p.n_heads + g * G) * HD + i] = a * sh.inv[h];
      }
      // the weights of this CTA's tokens; inv has the probabilities' 2^kLift
      for (int t = jt; t < u.have; t += 128) {
        float w = 0.0f;
#pragma unroll
        for (int h = 0; h < G; ++h) w = fmaf(ex2(sc[h * cap + t] - sh.M[h] + kLift), sh.inv[h], w);
        const int b = ids[t >> 4];
        if (b >= 0) atomicAdd(p.c.weights + ((size_t)b * p.c.n_kv_heads + g) * 16 + (t & 15), w);
      }
      mbar_arrive(&sh.part_free[buf]);
      meet();  // ids, M and inv are free
      u = then;
      then = later;
      if (++buf3 == 3) {
        buf3 = 0;
        phase3 ^= 1;
      }
    }
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_free(tmem, 64);
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (!ok) __nanosleep(1000000);  // what this CTA no longer waited for may be on its way
}

template <int HD, int G>
cudaError_t launch_t(const DecodeWeightsParams& p, cudaStream_t st) {
  using Lay = Layout<HD>;
  constexpr int kMaxSmem = 226 * 1024 - (int)sizeof(Shared<HD, G>);  // of 227 KB, in whole KB
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  static std::atomic<int> held[64][kMaxCluster + 1];  // CTAs that the device holds, one per SM, by cluster size
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_attention_weights<HD, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_attention_weights<HD, G>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int k = 1; k <= kMaxCluster && e == cudaSuccess; ++k) {
      int clusters = 0;
      attr[0].val.clusterDim.x = k;
      cfg.gridDim = dim3(1024 * k);
      cfg.dynamicSmemBytes = kMaxSmem;
      if (cudaOccupancyMaxActiveClusters(&clusters, k_attention_weights<HD, G>, &cfg) != cudaSuccess) {
        cudaGetLastError();  // a size that this device does not take is not used
        clusters = 0;
      }
      held[dev][k].store(clusters * k, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) return e;
    prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  Maps maps;
  // a block at once, as groups of 8 rows: [group][half][8][64]
  const uint64_t cd[4] = {64, 8, (uint64_t)Lay::H, (uint64_t)p.c.n_blocks * p.c.n_kv_heads * 2},
                 cs[3] = {(uint64_t)HD * 2, 128, (uint64_t)HD * 16};
  const uint32_t cb[4] = {64, 8, (uint32_t)Lay::H, 2};
  if (!encode_tensor_map(&maps.k, false, 4, p.c.k, cd, cs, cb) || !encode_tensor_map(&maps.v, false, 4, p.c.v, cd, cs, cb))
    return cudaErrorInvalidValue;
  // The cluster size with the least estimated time, in us: 5.5 for launch, first loads
  // and the last join, and for every round of units the larger of its blocks'
  // bytes at the SMs' share of the memory's bandwidth (44.5 GB/s each) and of its
  // tiles one after another (1.0 each, more where fewer than five tiles of the ring are
  // left beside the scores).  A last round that is not full is a little shorter.  The
  // GPCs (of up to 20 SMs) decide how many clusters fit.  Scores are double-buffered
  // where the ring keeps five tiles.  Fitted to 15 shapes with C = 1 .. 12, of which
  // it finds the best C or one 1% slower on average; measured with 8 kv heads
  // of 128, 4 query heads each: 32 sequences of 2176 tokens with C = 1, 2, 3, 4, 8: 58,
  // 58, 57, 60, 80 us; 64 of 300 with 1, 2, 4: 26, 35, 59; 32 of 8192 with 2, 4, 8, 12:
  // 204, 197, 186, 225; one of 2113 with 1, 4, 9, 12: 22.6, 11.3, 8.9, 9.4.
  const int units = p.batch * p.c.n_kv_heads, nb = (p.c.max_ctx + 15) / 16;
  int C = 0, grid = 0, ns = 0, buffers = 0;
  double least = 0.0;
  for (int k = 1; k <= kMaxCluster; ++k) {
    const int one = held[dev][k].load(std::memory_order_relaxed);
    if (one < 1 || (C > 0 && nb <= 8 * (k - 1))) continue;
    const int clusters = std::min(units, one / k), rounds = (units + clusters - 1) / clusters, each = (nb + k - 1) / k;
    auto room = [&](int copies) {
      const int64_t left = kMaxSmem - 1024 - (int64_t)Parts<HD, G>::bytes(each * 16, copies);
      return left < 0 ? 0 : std::min<int>(Lay::kMost, (int)(left / (int)Lay::kTile));
    };
    const int copies = rounds > 1 && room(2) >= 5 ? 2 : 1, fit = room(copies), tiles = (each + 7) / 8;
    if (fit < 3) continue;
    const double live = (double)clusters * k / sms, some = 0.8 * rounds + 0.2 * units / clusters;
    const double stream = each * live * (2.0 * Lay::kTile / 8 / 44.5e3) + 2.0;
    const double chain = tiles * (1.0 + 0.5 * std::max(0, 5 - fit)) + 1.3;
    const double t = 5.5 + some * std::max(stream, chain);
    if (C == 0 || t < least) {
      C = k;
      grid = clusters * k;
      ns = rounds > 1 ? fit : std::min(fit, std::max(3, 2 * tiles));
      buffers = copies;
      least = t;
    }
  }
  if (C == 0) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.dynamicSmemBytes = 1024 + ns * Lay::kTile + Parts<HD, G>::bytes((nb + C - 1) / C * 16, buffers);
  cfg.stream = st;
  attr[0].val.clusterDim.x = C;
  return cudaLaunchKernelEx(&cfg, k_attention_weights<HD, G>, p, maps, make_exponent(HD).c, ns, buffers);
}

}  // namespace

cudaError_t launch_attention_weights(const DecodeWeightsParams& p, cudaStream_t st) {
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

}  // namespace ee
