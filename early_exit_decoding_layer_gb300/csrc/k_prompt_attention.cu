// Causal attention of packed prompt rows over the paged cache, on the tensor
// cores (tcgen05.mma, fp32 accumulators in tensor memory).
//
// A CTA owns 256 rows of S = Q K^T for one kv head: row r is query head r % G of
// the group at the prompt's position i0 + r / G, so that one read of K and V
// serves the whole group.  The rows are two M = 128 tiles with a softmax
// warpgroup each; while one is busy with its probabilities the tensor core works
// for the other:
//   warp 9 (one thread)  O_t += P_t V_j, then S_t = Q_t K_{j + 1}^T, t = 0, 1 in turn
//   warps 4t .. 4t + 3   a thread per row: S_t to registers, the running maximum
//                        and sum, P_t = exp2(c S - c m) as fp16 over S_t's columns;
//                        S_t of a step also says that the K and V before are free
//   warp 8               Q, and K and V tiles of 128 keys by TMA, one copy per 16-slot
//                        block and 64 columns, into a ring of NST tiles
//   warp 10              waits for K and V tiles in warp 9's place, and looks V over
//   warp 11              finds the CTA's next units of work
// A CTA goes from unit to unit (tile of rows, kv head), its loads and first products
// ahead of the softmax warps.
//
// Maximum and sum run along the keys as in online softmax (Milakov and Gimelshein,
// 2018).  The maximum may lag behind by up to 8 (in log2): then P is at most 2^8
// instead of 1, which fp16 holds as exactly, and O, in tensor memory, is
// rescaled only when a row's maximum has grown by more than that.  The sum is
// kept in fp32 from the unrounded P; rounding P to fp16 (2^-11 of it) is the
// price of feeding the second product to the tensor core (a second fp16 part would
// add half of the products' time again).  o is fp16 itself, which alone is an error of
// 2.05e-4 (2-norm); with P's it is 2.2e-4 where a few tokens have most of the weight, and
// 2.95e-4 where 16384 random ones share it.
//
// Tiles that some row does not see whole are masked by comparing positions, so
// a NaN score is dropped as any other.  A NaN or infinity in V times a zero
// probability would not be: in those tiles warp 10 replaces such values by
// zero in shared memory, and where they stand for tokens of the sequence the
// rows that see them get them added at the end.
//
// Few rows over many keys (a chunk behind a long prefix): the keys are split over
// the CTAs of a cluster, which join their (O, m, l) through distributed shared
// memory in rank order.  No scratch, no atomics.
//
// Bound: the tensor core (4 hd flops per visible pair and query head); 16384 tokens
// of 32/8 heads, hd 128, take 1.56 ms, 1410 TFLOP/s, of which a step of 128 keys
// is 3200 cycles for 2190 of products: softmax (1370) and a tile's two products
// (1240) follow each other, and the two tiles overlap but for that.  256 rows per CTA
// and not 128: K and V then come from L2 at half the rate, which would be 17
// TB/s at the tensor core's peak.  32 packed prompts of 256 to 2048: 0.37 ms.
#include <cooperative_groups.h>
#include <math.h>

#include <atomic>

#include "ee_cache_ops.cuh"
#include "ee_tcgen05.cuh"

namespace cg = cooperative_groups;

namespace ee {
namespace {

constexpr int kRows = 256;     // rows of S per CTA: two tiles of 128
constexpr int kKeys = 128;     // keys per step
constexpr int kThreads = 384;  // two softmax warpgroups, TMA, MMA, landed tiles, units
constexpr int kMaxCluster = 6;
constexpr int kRegs = 168, kRegsSoftmax = 208, kRegsSingle = 88;  // at launch, and after
static_assert(256 * kRegsSoftmax + 128 * kRegsSingle <= kThreads * kRegs, "no more than the launch has");

template <int HD, bool SPLIT>
struct Shape {
  static constexpr int H = HD / 64;                       // 64-column halves
  static constexpr uint32_t kTile = 128 * HD * 2;         // a Q, K or V tile
  static constexpr uint32_t kHalf = 128 * 128;            // one 64-column half of it
  // ring tiles: as many as fit.  A tile's way from L2 takes about as long as a step, and
  // with four of them one step in two waited for V some 500 cycles.
  static constexpr int NST = HD == 128 ? (SPLIT ? 4 : 5) : 9;
  static constexpr size_t kSmem = 1024 + (2 + NST) * (size_t)kTile;
  static constexpr int kPad = HD + 4;                     // floats per joined row
  static_assert(!SPLIT || (size_t)kRows * kPad * 4 <= (2 + NST) * (size_t)kTile, "the join reuses the tiles' space");
};

struct Maps {
  CUtensorMap q, k, v;
};

// log of the sum of exp(s / sqrt(hd)), from its sum l relative to the score m.
EE_DEV float log_sum(float m, float l, const Exponent& ex) {
  return l == 0.0f ? -INFINITY : fmaf(m, ex.unit_hi, fmaf(m, ex.unit_lo, logf(l)));
}

// o is a mean of fp16 values and no larger than they are.  P's rounding may take it past the
// largest one by up to 2^-11 of it, which would be infinite in fp16.
constexpr float kMostHalf = 65504.0f;
EE_DEV float within_half(float y) {
  return fabsf(y) > kMostHalf && fabsf(y) < INFINITY ? copysignf(kMostHalf, y) : y;
}

// The work of one CTA on one (tile of rows, kv head): key tiles [ka, kb) of 128,
// of which row tile t takes the first n[t]; those from jm[t] on are not seen whole by
// every row of it.
struct Unit {
  PromptTile tl;
  int g, off, ka, kb, n[2], jm[2];
};

constexpr int kUnits = 4;  // units known ahead

// What only the join needs.
template <bool SPLIT>
struct Join {};
template <>
struct Join<true> {
  float m[kRows], l[kRows];           // of the CTA's share of the keys
  float fac[kMaxCluster][kRows / 2];  // what a rank's O counts in a row
};

template <int HD, bool SPLIT>
struct Shared : Join<SPLIT> {
  static constexpr int NST = Shape<HD, SPLIT>::NST;
  uint64_t q_full, q_free, kv_full[NST], kv_empty[NST], s_full[2], p_ready[2], o_done[2];
  uint64_t unit_full[kUnits], unit_free[kUnits];
  uint64_t drained;  // every MMA issued is over
  Unit unit[kUnits];
  uint32_t tmem;
  int bad_v[8];  // [unit & 7]: the last unit in which a non-finite V value was replaced
};

template <int G>
EE_DEV Unit make_unit(const PromptTile& tl, int g, int split, int nsplit) {
  constexpr int kPos = kRows / G;
  Unit u;
  u.tl = tl;
  u.g = g;
  u.off = tl.sq.ctx - tl.sq.n;  // position of row 0
  int nt[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r0 = tl.i0 + t * (kPos / 2), r1 = min(tl.sq.n, r0 + kPos / 2);
    nt[t] = r1 > r0 ? max(0, u.off + r1 + kKeys - 1) / kKeys : 0;
    u.jm[t] = max(0, u.off + r0 + 1) / kKeys;
  }
  const int all = max(nt[0], nt[1]), each = (all + nsplit - 1) / nsplit;
  u.ka = min(all, split * each);
  u.kb = min(all, u.ka + each);
#pragma unroll
  for (int t = 0; t < 2; ++t) u.n[t] = max(0, min(nt[t], u.kb) - u.ka);
  return u;
}

template <int HD, int G, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_prompt_attention(const PromptParams p, const __grid_constant__ Maps maps, const Exponent ex) {
  using S = Shape<HD, SPLIT>;
  constexpr int kPos = kRows / G;  // positions per CTA
  const float c = ex.c;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<HD, SPLIT> sh;
  uint8_t* tiles = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nsplit = SPLIT ? (int)cg::this_cluster().num_blocks() : 1;
  const int split = SPLIT ? (int)cg::this_cluster().block_rank() : 0;
  if (tid == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_free, 1);
    mbar_init(&sh.drained, 1);
    for (int i = 0; i < S::NST; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_ready[t], 129);  // its warpgroup, and V and K landed
      mbar_init(&sh.o_done[t], 1);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&sh.unit_full[i], 1);
      mbar_init(&sh.unit_free[i], 11);  // every warp but the one that finds them
    }
    for (int i = 0; i < 8; ++i) sh.bad_v[i] = -1;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t q_s = smem_addr(tiles), kv_s = q_s + 2 * S::kTile;
  // tensor memory: S_t (128 columns, P_t over its first 64), then O_t
  auto s_col = [&](int t) { return tmem + t * 128; };
  auto o_col = [&](int t) { return tmem + 256 + t * HD; };
  // Ring items count on over the units: item base + 2 j is K of the unit's key tile
  // ka + j, item base + 2 j + 1 its V.
  auto stage = [&](int i) { return i % S::NST; };
  auto phase = [&](int i) { return (uint32_t)(i / S::NST) & 1; };

  // Unit i of this CTA, found by warp 11; s = -1: no more.
  auto unit_at = [&](int i) {
    Unit u;
    u.tl.s = -1;
    if (warp_wait(&sh.unit_full[i % kUnits], (i / kUnits) & 1, p.c.err, DERR_FULL_WAIT)) {
      u = sh.unit[i % kUnits];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.unit_free[i % kUnits]);
    }
    return u;
  };

  // Registers go from the four single warps to the softmax warps, which hold a row of
  // S: 128 x 88 + 256 x 208 is what 384 threads are launched with at 168 each
  // (launch_t checks that).
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsSingle));
  if (warp == 11) {
    // Not split: a CTA takes units until there are none, every second round in the
    // opposite order, which evens out what the falling sizes leave uneven.
    // Split: a cluster has one.
    PromptIndex index;
    index.init(p, kPos);
    for (int i = 0;; ++i) {
      int at = blockIdx.x / nsplit;
      if (!SPLIT) at = i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      PromptTile tl = {-1, 0, {0, 0, 0}};
      if (!SPLIT || i == 0) tl = index.find(at / p.c.n_kv_heads);
      const Unit u = make_unit<G>(tl, at % p.c.n_kv_heads, split, nsplit);
      if (i >= kUnits && !warp_wait(&sh.unit_free[i % kUnits], (i / kUnits - 1) & 1, p.c.err, DERR_EMPTY_WAIT)) break;
      if (lane == 0) {
        sh.unit[i % kUnits] = u;
        mbar_arrive(&sh.unit_full[i % kUnits]);
      }
      __syncwarp();
      if (tl.s < 0) break;
    }
  } else if (warp == 8) {
    Unit u = unit_at(0);
    const int b8 = lane & 7, half = lane >> 3;
    int issued = 0, loads = 0;
    bool ok = true;
    for (int i = 0; u.tl.s >= 0 && ok; u = unit_at(++i)) {
      const int nblk = (u.tl.sq.ctx + 15) >> 4;
      const int32_t* bt = p.c.table + (int64_t)u.tl.s * p.c.table_stride;
      auto block_id = [&](int j) {  // of block b8 of key tile j
        const int b = j * 8 + b8;
        int id = b < nblk && j < u.kb ? bt[b] : 0;
        if (id < 0 || id >= p.c.n_blocks) {
          report(p.c.err, EE_DERR_BLOCK);
          id = 0;
        }
        return id;
      };
      int id = block_id(u.ka);
      // a unit whose rows see anything has its Q loaded; q_free: the products of the
      // one before have read theirs
      if (u.kb > u.ka) {
        if (loads > 0) ok = warp_wait(&sh.q_free, (loads - 1) & 1, p.c.err, DERR_EMPTY_WAIT);
        loads += ok;
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full, (u.n[0] > 0 ? S::kTile : 0) + (u.n[1] > 0 ? S::kTile : 0));
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (u.n[t] > 0)
              for (int h = 0; h < S::H; ++h)
                tma_load_3d(q_s + t * S::kTile + h * S::kHalf, &maps.q, h * 64, u.g * G,
                            u.tl.sq.first + u.tl.i0 + t * (kPos / 2), &sh.q_full);
        }
        __syncwarp();
      }
      for (int j = u.ka; j < u.kb && ok; ++j) {
        const int next = block_id(j + 1), here = min(8, nblk - j * 8);
        for (int kv = 0; kv < 2; ++kv, ++issued) {
          const int st = stage(issued);
          if (issued >= S::NST) ok = warp_wait(&sh.kv_empty[st], phase(issued - S::NST), p.c.err, DERR_EMPTY_WAIT);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[st], (uint32_t)here * 16 * HD * 2);
          __syncwarp();
          if (half < S::H && b8 < here)
            tma_load_2d(kv_s + st * S::kTile + half * S::kHalf + b8 * 2048, kv ? &maps.v : &maps.k, half * 64,
                        (id * p.c.n_kv_heads + u.g) * 16, &sh.kv_full[st]);
        }
        id = next;
      }
    }
    // Copies land before the CTA ends, whichever warp gave up (where none did, they have).
    for (int i = max(0, issued - S::NST); i < issued; ++i)
      mbar_wait_bounded(&sh.kv_full[stage(i)], phase(i), p.c.err, DERR_DRAIN_WAIT);
    if (loads > 0) mbar_wait_bounded(&sh.q_full, (loads - 1) & 1, p.c.err, DERR_DRAIN_WAIT);
  } else if (warp == 9) {
    // One thread issues every MMA.  The tensor core takes an MMA from it when it
    // starts on it, so what the thread does between two products costs the
    // tensor core time: a step's O and next S products of a tile go out together,
    // each wait that can be left to another warp is, and commits are few.  The
    // commit behind S_t(j + 1) also says that O_t has P_t V_j.
    Unit u = unit_at(0);
    constexpr uint32_t id_qk = instr_desc(0, kKeys, 128), id_pv = instr_desc(0, HD, 128, true);
    int base = 0, steps[2] = {0, 0}, loads = 0;
    bool ok = true;
    for (int i = 0; u.tl.s >= 0 && ok; u = unit_at(++i)) {
      const int nk = u.kb - u.ka;
      if (lane == 0 && nk > 0) {
        auto qk = [&](int t, int j) {
          const uint32_t a = q_s + t * S::kTile, b = kv_s + stage(base + 2 * j) * S::kTile;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t o = (kk >> 2) * S::kHalf + (kk & 3) * 32;
            mma_f16(s_col(t), smem_desc_sw128(a + o), smem_desc_sw128(b + o), id_qk, kk > 0);
          }
          mma_commit(&sh.s_full[t]);
        };
        ok = mbar_wait_bounded(&sh.q_full, loads & 1, p.c.err, DERR_FULL_WAIT) &&
             mbar_wait_bounded(&sh.kv_full[stage(base)], phase(base), p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        if (ok && u.n[0] > 0) qk(0, 0);
        if (ok && u.n[1] > 0) qk(1, 0);
        for (int j = 0; j < nk && ok; ++j) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int n = u.n[t];
            if (j < n) {
              // P_t(j) is in tensor memory, V_j and K_{j + 1} have landed
              if (!(ok = mbar_wait_bounded(&sh.p_ready[t], steps[t] & 1, p.c.err, DERR_FULL_WAIT))) break;
              ++steps[t];
              tc_fence_after();
              const uint32_t b = kv_s + stage(base + 2 * j + 1) * S::kTile;
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_f16_ta(o_col(t), s_col(t) + kk * 8, smem_desc_sw128_mn(b + kk * 2048, S::kHalf), id_pv,
                           j > 0 || kk > 0);
              if (j + 1 < n) qk(t, j + 1);
              else mma_commit(&sh.o_done[t]);
            }
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      base += 2 * nk;
      loads += nk > 0;
    }
    if (lane == 0) {  // and so are the products, before tensor memory is given back
      mma_commit(&sh.drained);
      mbar_wait_bounded(&sh.drained, 0, p.c.err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else if (warp == 10) {
    // Waits for V_j and K_{j + 1} on behalf of the MMA thread: P_t(j)'s barriers
    // count this warp's arrival too.  In tiles that are masked for some row, V
    // values that are not finite become 0 before the product reads them.
    Unit u = unit_at(0);
    int base = 0, steps[2] = {0, 0};
    bool ok = true;
    for (int i = 0; u.tl.s >= 0 && ok; u = unit_at(++i)) {
      const int nk = u.kb - u.ka;
      for (int j = 0; j < nk && ok; ++j) {
        const int v = base + 2 * j + 1;
        ok = warp_wait(&sh.kv_full[stage(v)], phase(v), p.c.err, DERR_FULL_WAIT);
        if (ok && u.ka + j >= min(u.jm[0], u.jm[1])) {
          uint8_t* vt = tiles + 2 * S::kTile + stage(v) * S::kTile;
          const int chunks = (int)(S::kTile / 16) / 32;  // 16-byte chunks per lane
          uint32_t any = 0;
#pragma unroll 8
          for (int k = 0; k < chunks; ++k) {
            const uint4 x = *reinterpret_cast<const uint4*>(vt + (k * 32 + lane) * 16);
            any |= ((x.x & 0x7c007c00u) + 0x04000400u) | ((x.y & 0x7c007c00u) + 0x04000400u) |
                   ((x.z & 0x7c007c00u) + 0x04000400u) | ((x.w & 0x7c007c00u) + 0x04000400u);
          }
          if (__any_sync(0xffffffffu, any & 0x80008000u)) {
            bool fixed = false;
            for (int k = 0; k < chunks; ++k) {
              const int at = (k * 32 + lane) * 16;
              uint32_t w[4];
              *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(vt + at);
              bool hit = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((w[e] & 0x7c00u) == 0x7c00u) w[e] &= 0xffff0000u, hit = true;
                if ((w[e] & 0x7c000000u) == 0x7c000000u) w[e] &= 0x0000ffffu, hit = true;
              }
              if (hit) {
                *reinterpret_cast<uint4*>(vt + at) = make_uint4(w[0], w[1], w[2], w[3]);
                // rows of the tile are 128 bytes in each half
                if ((u.ka + j) * kKeys + (at % (int)S::kHalf) / 128 < u.tl.sq.ctx) fixed = true;
              }
            }
            if (__any_sync(0xffffffffu, fixed) && lane == 0) sh.bad_v[i & 7] = i;
            fence_proxy_async();
            __syncwarp();
          }
        }
        if (ok && j + 1 < nk) ok = warp_wait(&sh.kv_full[stage(v + 1)], phase(v + 1), p.c.err, DERR_FULL_WAIT);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || j >= u.n[t]) continue;
          // one phase of p_ready per step: the one before has to be over
          if (steps[t] > 0) ok = warp_wait(&sh.p_ready[t], (steps[t] - 1) & 1, p.c.err, DERR_FULL_WAIT);
          if (ok && lane == 0) mbar_arrive(&sh.p_ready[t]);
          ++steps[t];
        }
      }
      base += 2 * nk;
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, r = tid & 127;  // tile and row
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = s_col(t) + lane_base, o_at = o_col(t) + lane_base;
    Unit u = unit_at(0);
    int base = 0, steps = 0, ends = 0;
    bool ok = true;
    for (int i = 0; u.tl.s >= 0 && ok; u = unit_at(++i)) {
      const int n = u.n[t], nk = u.kb - u.ka;
      const int row = u.tl.i0 + t * (kPos / 2) + r / G;
      const bool valid = row < u.tl.sq.n;
      const int pos = valid ? u.off + row : -1;  // last key this row sees
      // the tile whose products come last in a step: n[1] >= n[0] or n[1] = 0
      const bool frees = r == 0 && t == (u.n[1] > 0 ? 1 : 0);
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < n && ok; ++j) {
        if (!(ok = warp_wait(&sh.s_full[t], steps & 1, p.c.err, DERR_FULL_WAIT))) break;
        ++steps;
        tc_fence_after();
        if (frees) {  // the tiles of the products before are free
          if (j > 0) mbar_arrive(&sh.kv_empty[stage(base + 2 * j - 1)]);
          mbar_arrive(&sh.kv_empty[stage(base + 2 * j)]);
        }
        if (frees && j == n - 1) mbar_arrive(&sh.q_free);  // the last product with Q, of both tiles
        const bool masked = u.ka + j >= u.jm[t];
        uint32_t s[kKeys], ph[kKeys / 2];
        auto load = [&]() {
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s + 32 * i);
          tmem_wait_ld();
          tmem_pin<kKeys>(s);
          if (masked) {
            const int lim = pos - (u.ka + j) * kKeys;
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
              if (i > lim) s[i] = 0xff800000u;  // -inf
          }
        };
        auto maximum = [&]() {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kKeys; i += 8)
#pragma unroll
            for (int w = 0; w < 4; ++w)
              mx[w] = max3(mx[w], __uint_as_float(s[i + 2 * w]), __uint_as_float(s[i + 2 * w + 1]));
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        };
        // P of all keys into ph, returns their sum
        auto exponentials = [&]() {
          // a row that has seen nothing yet has m = -inf: its P is 0
          const float mc = m == -INFINITY ? 0.0f : m * c;
          const uint64_t c2 = pack2(c, c), nm2 = pack2(-mc, -mc);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < kKeys; i += 2) {
            const float2 x = unpack2(fma2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, nm2));
            const float e0 = ex2(x.x), e1 = ex2(x.y);
            sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(e0, e1));
            const __half2 h = __floats2half2_rn(e0, e1);
            ph[i >> 1] = *reinterpret_cast<const uint32_t*>(&h);
          }
          const float2 st = unpack2(add2(sum[0], sum[1]));
          return st.x + st.y;
        };
        load();
        const float mt = maximum();
        if (j == 0) {
          m = mt;
        } else if (__any_sync(0xffffffffu, (mt - m) * c > 8.0f)) {
          // some row's maximum has grown too far: this warp's rows of O and l go over to
          // the new maxima (O has every product before: S_t(j) came after)
          const float mn = fmaxf(m, mt);
          const float a = m == mn ? 1.0f : ex2((m - mn) * c);
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
        l += exponentials();
#pragma unroll
        for (int i = 0; i < kKeys / 2; i += 16) tmem_st16(s_at + i, ph + i);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.p_ready[t]);
      }
      if (ok && n > 0) ok = warp_wait(&sh.o_done[t], ends & 1, p.c.err, DERR_FULL_WAIT);
      ends += n > 0;
      tc_fence_after();
      if (frees && nk > 0) mbar_arrive(&sh.kv_empty[stage(base + 2 * nk - 1)]);
      // for the join, which reuses the tiles' space, the other row tile has to be done too
      if (SPLIT && ok && u.n[1 - t] > 0) ok = warp_wait(&sh.o_done[1 - t], 0, p.c.err, DERR_FULL_WAIT);
      const bool bad = sh.bad_v[i & 7] == i;
      const int jm = min(u.jm[0], u.jm[1]);
      const int head = u.g * G + r % G;
      const float il = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // NaN stays
      uint16_t* orow = p.o + (int64_t)(u.tl.sq.first + row) * p.o_stride + head * HD;
      float* jrow = reinterpret_cast<float*>(tiles) + (size_t)(t * 128 + r) * S::kPad;
      if (SPLIT) {
#pragma unroll 1
        for (int i = 0; i < HD; i += 32) {
          uint32_t o[32];
          tmem_ld32(o_at + i, o);
          tmem_wait_ld();
          tmem_pin<32>(o);
#pragma unroll
          for (int w = 0; w < 32; w += 4)
            *reinterpret_cast<uint4*>(jrow + i + w) =
                n > 0 ? make_uint4(o[w], o[w + 1], o[w + 2], o[w + 3]) : make_uint4(0, 0, 0, 0);
        }
      } else if (ok) {
        // Two neighbouring lanes write their rows together, 32 bytes each side by side: a
        // thread that stores its own row alone touches a line per lane.
        const bool wide = ((uintptr_t)p.o & 31) == 0 && (p.o_stride & 15) == 0, odd = lane & 1;
        uint16_t* other = reinterpret_cast<uint16_t*>(__shfl_xor_sync(0xffffffffu, (unsigned long long)orow, 1));
        const bool other_valid = __shfl_xor_sync(0xffffffffu, valid, 1);
        uint16_t* row_a = (odd ? other : orow) + (odd ? 16 : 0);  // of the even lane
        uint16_t* row_b = (odd ? orow : other) + (odd ? 16 : 0);
        const bool a_valid = odd ? other_valid : valid, b_valid = odd ? valid : other_valid;
        const uint64_t il2 = pack2(il, il);
        float most = 0.0f;
#pragma unroll 1
        for (int i = 0; i < HD; i += 32) {
          uint32_t o[32], h[16], x[8];
          tmem_ld32(o_at + i, o);
          tmem_wait_ld();
          tmem_pin<32>(o);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 y = unpack2(mul2(pack2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), il2));
            most = max3(most, fabsf(y.x), fabsf(y.y));
            const __half2 z = __floats2half2_rn(y.x, y.y);
            h[k] = n > 0 ? *reinterpret_cast<const uint32_t*>(&z) : 0;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = __shfl_xor_sync(0xffffffffu, odd ? h[k] : h[8 + k], 1);
          uint32_t ra[8], rb[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            ra[k] = odd ? x[k] : h[k];
            rb[k] = odd ? h[8 + k] : x[k];
          }
          if (wide) {
            if (a_valid) st_global_v8(row_a + i, ra);
            if (b_valid) st_global_v8(row_b + i, rb);
          } else {
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
              if (a_valid) *reinterpret_cast<uint4*>(row_a + i + 2 * k) = make_uint4(ra[k], ra[k + 1], ra[k + 2], ra[k + 3]);
              if (b_valid) *reinterpret_cast<uint4*>(row_b + i + 2 * k) = make_uint4(rb[k], rb[k + 1], rb[k + 2], rb[k + 3]);
            }
          }
        }
        __syncwarp();
        if (__any_sync(0xffffffffu, n > 0 && most > kMostHalf)) {  // rare, as below
#pragma unroll 1
          for (int i = 0; i < HD; i += 16) {
            uint32_t o[16];
            tmem_ld16(o_at + i, o);
            tmem_wait_ld();
            tmem_pin<16>(o);
#pragma unroll
            for (int w = 0; w < 16; ++w) {
              const float y = __uint_as_float(o[w]) * il, z = within_half(y);
              if (valid && z != y) orow[i + w] = float_to_half_bits(z);  // (a NaN differs too, and stays)
            }
          }
        }
      }
      if (bad && ok && valid) {
        // the values taken out of V, for the rows that see them (rare: kept out of the
        // loop above, whose code is fetched anew for every unit)
        const int end = min(pos, u.kb * kKeys - 1);
#pragma unroll 1
        for (int tok = max(jm, u.ka) * kKeys; tok <= end; ++tok) {
          bool bok;
          const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, u.tl.s, tok, nullptr, &bok);
          const uint16_t* v = p.c.v + (((size_t)b * p.c.n_kv_heads + u.g) * 16 + (tok & 15)) * HD;
#pragma unroll 1
          for (int w = 0; w < HD; ++w) {
            if ((v[w] & 0x7c00u) != 0x7c00u) continue;
            const float x = __half2float(__ushort_as_half(v[w]));
            if (SPLIT) jrow[w] += x;
            else orow[w] = float_to_half_bits(__half2float(__ushort_as_half(orow[w])) + x);
          }
        }
      }
      if constexpr (SPLIT) {
        sh.m[t * 128 + r] = m;
        sh.l[t * 128 + r] = l;
      } else if (valid && ok && p.lse) {
        p.lse[(size_t)head * p.total_q + u.tl.sq.first + row] = log_sum(m, l, ex);
      }
      tc_fence_before();
      base += 2 * nk;
    }
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
  if constexpr (SPLIT) {
    // Rank r joins rows r, r + nsplit, ...: every rank's (O, m, l) in rank order.
    // First what each rank's O counts in a row (eight lanes per row, one per
    // rank), then the rows.  Short code rather than many reads in flight: it runs
    // once, and fetching it counts.
    cg::cluster_group cl = cg::this_cluster();
    const Unit u = sh.unit[0];
    cl.sync();
    const int rows = u.tl.s < 0 ? 0 : min(kRows, (u.tl.sq.n - u.tl.i0) * G);
    const int mine = rows > split ? (rows - split + nsplit - 1) / nsplit : 0;
#pragma unroll 1
    for (int i0 = 0; i0 < mine; i0 += kThreads / 8) {
      const int i = i0 + tid / 8, k = tid & 7, r = split + nsplit * i;
      const Shared<HD, SPLIT>* o = cl.map_shared_rank(&sh, k < nsplit ? k : split);
      const bool has = k < nsplit && i < mine;
      const float m = has ? o->m[r] : -INFINITY, l = has ? o->l[r] : 0.0f;
      float M = m;
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      const float a = l == 0.0f ? 0.0f : m == M ? 1.0f : ex2((m - M) * c);  // 0: saw nothing
      float sum = a * l;  // a may have gone to 0: a NaN stays
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      if (has) {
        sh.fac[k][i] = a * (sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum));  // NaN stays
        const int row = u.tl.i0 + r / G, head = u.g * G + r % G;
        if (k == 0 && p.lse) p.lse[(size_t)head * p.total_q + u.tl.sq.first + row] = log_sum(M, sum, ex);
      }
    }
    __syncthreads();
    constexpr int L = HD / 4;  // threads per row
    const int col = (tid % L) * 4;
#pragma unroll 1
    for (int i = tid / L; i < mine; i += kThreads / L) {
      const int r = split + nsplit * i;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int k0 = 0; k0 < nsplit; k0 += 4) {
        float4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = *reinterpret_cast<const float4*>(
              cl.map_shared_rank(reinterpret_cast<float*>(tiles), k0 + k < nsplit ? k0 + k : split) + (size_t)r * S::kPad + col);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k0 + k < nsplit) {
            // a rank that saw nothing has O = 0; one that counts 0 for its small scores may
            // have an infinity or NaN, which stays
            const float a = sh.fac[k0 + k][i];
            o.x = fmaf(a, x[k].x, o.x);
            o.y = fmaf(a, x[k].y, o.y);
            o.z = fmaf(a, x[k].z, o.z);
            o.w = fmaf(a, x[k].w, o.w);
          }
        }
      }
      const int row = u.tl.i0 + r / G, head = u.g * G + r % G;
      const __half2 h0 = __floats2half2_rn(within_half(o.x), within_half(o.y)),
                    h1 = __floats2half2_rn(within_half(o.z), within_half(o.w));
      *reinterpret_cast<uint2*>(p.o + (int64_t)(u.tl.sq.first + row) * p.o_stride + head * HD + col) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    }
    cl.sync();  // nobody leaves while its memory is read
  }
}

template <int HD, int G>
cudaError_t launch_t(const PromptParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_prompt_attention<HD, G, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shape<HD, false>::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_prompt_attention<HD, G, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Shape<HD, true>::kSmem);
    // the exchange of registers above counts on the launch's share
    for (const void* f : {(const void*)k_prompt_attention<HD, G, false>, (const void*)k_prompt_attention<HD, G, true>}) {
      cudaFuncAttributes at;
      if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, f);
      if (e == cudaSuccess && at.numRegs != kRegs) e = cudaErrorInvalidConfiguration;
    }
    if (e != cudaSuccess) return e;
    if (dev < 64) prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Maps maps;
  const uint64_t qd[3] = {(uint64_t)HD, (uint64_t)p.n_heads, (uint64_t)p.total_q};
  const uint64_t qs[2] = {(uint64_t)HD * 2, (uint64_t)p.q_stride * 2};
  const uint32_t qb[3] = {64, (uint32_t)G, 128 / (uint32_t)G};
  const uint64_t cd[2] = {(uint64_t)HD, (uint64_t)p.c.n_blocks * p.c.n_kv_heads * 16}, cs[1] = {(uint64_t)HD * 2};
  const uint32_t cb[2] = {64, 16};
  if (!encode_tensor_map(&maps.q, false, 3, p.q, qd, qs, qb) || !encode_tensor_map(&maps.k, false, 2, p.c.k, cd, cs, cb) ||
      !encode_tensor_map(&maps.v, false, 2, p.c.v, cd, cs, cb))
    return cudaErrorInvalidValue;
  const Exponent ex = make_exponent(HD);
  // At most this many tiles: each sequence may leave one unfilled.  Where they leave
  // SMs idle the keys are split, as long as a CTA keeps some 2.5 key tiles: 60 rows
  // of 64/8 heads, hd 128, behind 16000 tokens take 236 us on 16 CTAs and 53 us on
  // 96; 512 rows of 32/8 heads, hd 64, 12.3 us unsplit and 14.5 us split in two.
  // Clusters of 8 were slower than of 6 (84 us): a GPC's 18 or 19 free SMs hold
  // three of 6 and only two of 8.
  const int64_t units = ((int64_t)p.total_q * G / kRows + p.n_seqs) * p.c.n_kv_heads;
  const int steps = (p.c.max_ctx + kKeys - 1) / kKeys;
  int split = 1;
  while (split < kMaxCluster && units * (split + 1) <= sms && 2 * steps >= 5 * (split + 1)) ++split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(split > 1 ? units * split : units < sms ? units : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = split > 1 ? Shape<HD, true>::kSmem : Shape<HD, false>::kSmem;
  cfg.stream = st;
  if (split == 1) return cudaLaunchKernelEx(&cfg, k_prompt_attention<HD, G, false>, p, maps, ex);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_prompt_attention<HD, G, true>, p, maps, ex);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptParams& p, cudaStream_t st) {
  const int G = p.n_heads / p.c.n_kv_heads, hd = p.c.head_dim;
#define EE_PROMPT_CASE(HD_, G_) \
  if (hd == HD_ && G == G_) return launch_t<HD_, G_>(p, st);
  EE_PROMPT_CASE(64, 1)
  EE_PROMPT_CASE(64, 2)
  EE_PROMPT_CASE(64, 4)
  EE_PROMPT_CASE(64, 8)
  EE_PROMPT_CASE(128, 1)
  EE_PROMPT_CASE(128, 2)
  EE_PROMPT_CASE(128, 4)
  EE_PROMPT_CASE(128, 8)
#undef EE_PROMPT_CASE
  return cudaErrorInvalidValue;
}

}  // namespace ee
