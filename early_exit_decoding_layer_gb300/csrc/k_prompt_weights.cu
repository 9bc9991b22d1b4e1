// What each cached token weighs in the attention of packed prompt rows, on the
// tensor cores: w[t] += sum over the rows (position, head of the group) that see
// t of exp(z_t - lse).
//
// The keys are the MMA's rows: S = K_tile Q^T gives every thread of a softmax
// warpgroup one key and, along its registers, 128 query rows, so the sum over
// the rows stays in the thread: no shuffles, and no second pass over anything.
// A CTA owns up to 256 keys of one kv head, two M = 128 tiles that stay in shared memory
// (one read of the queries serves both: with one tile their way from L2 was the
// limit); tiles of 128 query rows (128 / G positions x G heads) stream through
// a ring by TMA from the first row that sees a key:
//   warpgroup t          key tile t & 1, query tiles of parity t / 2: exp2(c S - f lse),
//                        summed; each has an S buffer in tensor memory
//   warp 16              TMA
//   warps 17, 18         (a thread of each) S = K Q_j^T, j even and odd
// Each tile's 128 terms are summed in four chains, and the tiles' sums with
// compensation, so that the error does not grow with the prompt's length.
//
// Bound: 8 sequences of 4096 tokens, 64/8 heads, hd 128: 908 us, 1210 TFLOP/s.  Nothing
// is full (tensor pipe 55%, exponentials 56%, issue slots 53%): with one S
// buffer each, a warpgroup's exponentials and its next product take turns.
//
// Few keys: the query tiles are dealt to the CTAs of a cluster, whose
// sums are joined through distributed shared memory in rank order.  A token's
// weight is added once per sequence and call (red.add: a block that several
// sequences share gets every part).
#include <cooperative_groups.h>
#include <math.h>

#include <atomic>

#include "ee_cache_ops.cuh"
#include "ee_tcgen05.cuh"

namespace cg = cooperative_groups;

namespace ee {
namespace {

constexpr int kTiles = 2;      // key tiles of 128 per CTA at most
constexpr int kCols = 128;     // query rows per tile
constexpr int kGroups = 4;     // softmax warpgroups, each with an S buffer of 128 tensor-memory columns
constexpr int kThreads = kGroups * 128 + 96;  // and TMA and two MMA warps
constexpr int kBuf = kGroups;
constexpr int kTma = kGroups * 4;  // warp; the two behind it issue the MMAs
constexpr int kMaxCluster = 4;

template <int HD>
struct Shape {
  static constexpr int H = HD / 64;
  static constexpr uint32_t kTile = 128 * HD * 2;
  static constexpr uint32_t kHalf = 128 * 128;
  static constexpr int NST = HD == 128 ? 4 : 6;
  static constexpr size_t kSmem = 1024 + (2 + NST) * (size_t)kTile;
};

struct Maps {
  CUtensorMap q, k;
};

struct Shared {
  uint64_t k_full, q_full[8], q_empty[8], s_full[kBuf], s_free[kBuf];
  uint64_t drained[2];  // every MMA of an issuing thread is over
  uint32_t tmem;
  alignas(16) float lse[kGroups][2][kCols];  // by warpgroup, two tiles
  uint2 odd[kGroups][kCols / 32];            // its columns of infinite (x) and NaN (y) lse, a bit each
  float sum[kGroups][128];
};

template <int HD, int G, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_prompt_weights(const PromptParams p, const __grid_constant__ Maps maps, const Exponent ex, const int key_tiles) {
  using S = Shape<HD>;
  constexpr int kPos = kCols / G;  // positions per query tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* tiles = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nsplit = SPLIT ? (int)cg::this_cluster().num_blocks() : 1;
  const int split = SPLIT ? (int)cg::this_cluster().block_rank() : 0;
  // first keys first: most rows see them
  const int unit = blockIdx.x / nsplit;
  const int g = unit % p.c.n_kv_heads, s = unit / p.c.n_kv_heads % p.n_seqs;
  const int key0 = unit / p.c.n_kv_heads / p.n_seqs * 128 * key_tiles;
  const PromptSeq sq = prompt_seq(p, s);
  const int off = sq.ctx - sq.n;
  const int first = max(0, key0 - off);  // first row that sees a key of the tile
  if (key0 >= sq.ctx || first >= sq.n) return;  // the whole cluster
  const int nh = key_tiles == 2 && key0 + 128 < sq.ctx ? 2 : 1;  // key tiles
  const int all = (sq.n - first + kPos - 1) / kPos;
  const int nq = (all - split + nsplit - 1) / nsplit;  // this CTA's: tiles split, split + nsplit, ...
  auto tile_row = [&](int j) { return first + (split + j * nsplit) * kPos; };

  if (tid == 0) {
    mbar_init(&sh.k_full, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.drained[i], 1);
    for (int i = 0; i < S::NST; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], nh);  // a warpgroup per key tile
    }
    for (int i = 0; i < kBuf; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], 128);
    }
    fence_mbar_init();
  }
  if (warp == kTma + 1) tmem_alloc(&sh.tmem, kBuf * kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t k_s = smem_addr(tiles), q_s = k_s + 2 * S::kTile;

  if (warp == kTma) {
    const int here = min(nh * 8, ((sq.ctx + 15) >> 4) - key0 / 16);  // blocks of the keys
    const int b16 = lane & 15, half = lane >> 4;
    if (nq > 0) {
      int id = b16 < here ? p.c.table[(int64_t)s * p.c.table_stride + key0 / 16 + b16] : 0;
      if (id < 0 || id >= p.c.n_blocks) {
        report(p.c.err, EE_DERR_BLOCK);
        id = 0;
      }
      if (lane == 0) mbar_arrive_expect_tx(&sh.k_full, (uint32_t)here * 16 * HD * 2);
      __syncwarp();
      if (half < S::H && b16 < here)
        tma_load_2d(k_s + (b16 >> 3) * S::kTile + half * S::kHalf + (b16 & 7) * 2048, &maps.k, half * 64,
                    (id * p.c.n_kv_heads + g) * 16, &sh.k_full);
    }
    if (lane == 0) {
      int issued = 0;
      for (int j = 0; j < nq; ++j, ++issued) {
        const int st = j % S::NST, pass = j / S::NST;
        if (pass > 0 && !mbar_wait_bounded(&sh.q_empty[st], (pass - 1) & 1, p.c.err, DERR_EMPTY_WAIT)) break;
        mbar_arrive_expect_tx(&sh.q_full[st], S::kTile);
        for (int h = 0; h < S::H; ++h)
          tma_load_3d(q_s + st * S::kTile + h * S::kHalf, &maps.q, h * 64, g * G, sq.first + tile_row(j), &sh.q_full[st]);
      }
      // Copies land before the CTA ends, whichever warp gave up (where none did, they have).
      if (nq > 0) mbar_wait_bounded(&sh.k_full, 0, p.c.err, DERR_DRAIN_WAIT);
      for (int i = max(0, issued - S::NST); i < issued; ++i)
        mbar_wait_bounded(&sh.q_full[i % S::NST], (i / S::NST) & 1, p.c.err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else if (warp > kTma) {
    // an issuing thread per warpgroup: what one does between two products falls into
    // the other's
    const int t = warp - kTma - 1;
    if (lane == 0 && t < nq) {
      constexpr uint32_t idesc = instr_desc(0, kCols, 128);
      bool ok = mbar_wait_bounded(&sh.k_full, 0, p.c.err, DERR_FULL_WAIT);
      for (int j = t; j < nq && ok; j += 2) {
        const int st = j % S::NST;
        const uint64_t q = smem_desc_sw128(q_s + st * S::kTile);
        ok = mbar_wait_bounded(&sh.q_full[st], (j / S::NST) & 1, p.c.err, DERR_FULL_WAIT);
#pragma unroll 1
        for (int h = 0; h < nh && ok; ++h) {
          const int b = 2 * t + h;
          const uint64_t a = smem_desc_sw128(k_s + h * S::kTile);
          if (j >= 2) ok = mbar_wait_bounded(&sh.s_free[b], (j / 2 - 1) & 1, p.c.err, DERR_EMPTY_WAIT);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * S::kHalf + (kk & 3) * 32) >> 4;
            mma_f16(tmem + b * kCols, a + o, q + o, idesc, kk > 0);
          }
          mma_commit(&sh.s_full[b]);
        }
      }
      // and so are the products, before tensor memory is given back
      mma_commit(&sh.drained[t]);
      mbar_wait_bounded(&sh.drained[t], 0, p.c.err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else {
    // warpgroup t: key tile t & 1, query tiles j = t / 2, t / 2 + 2, ..
    const int t = warp >> 2, r = tid & 127, keys = key0 + (t & 1) * 128, key = keys + r;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // Column r of a tile: its lse (a row of nobody is masked).  What becomes of it waits
    // until the next tile, when the load is over.  A column whose lse is infinite adds
    // nothing, whatever its scores are, and one with a NaN lse is NaN only for the keys that
    // it sees.  Neither comes out of c S - f lse, so a vote with the barrier that is there finds
    // tiles with such a column, which go their own way (with its conditions in the other
    // tiles' loop 8 x 4096 tokens took 938 us instead of 908).
    auto load_lse = [&](int j) {
      const int row = j < nq ? tile_row(j) + r / G : sq.n;
      return row < sq.n ? p.lse_in[(size_t)(g * G + r % G) * p.total_q + sq.first + row] : 0.0f;
    };
    float sum = 0.0f, comp = 0.0f, next = load_lse(t >> 1);
    const uint64_t c2 = pack2(ex.c, ex.c);
    bool ok = true;
    for (int j = t >> 1; j < ((t & 1) < nh ? nq : 0); j += 2) {
      float* ls = sh.lse[t][(j >> 1) & 1];
      const float now = next;
      ls[r] = -fmaf(now, ex.f_hi, now * ex.f_lo);  // in the exponent's unit
      next = load_lse(j + 2);
      // the other buffer was read two tiles ago, before the barrier of the last one
      int odd = !(fabsf(now) < INFINITY);
      asm volatile(
          "{ .reg .pred p, q; setp.ne.s32 p, %0, 0; barrier.cta.red.or.pred q, %1, 128, p; selp.s32 %0, 1, 0, q; }"
          : "+r"(odd)
          : "r"(1 + t)
          : "memory");
      if (odd) {
        const unsigned none = __ballot_sync(0xffffffffu, isinf(now)), nan = __ballot_sync(0xffffffffu, isnan(now));
        if (lane == 0) sh.odd[t][warp & 3] = make_uint2(none, nan);
        if (!(fabsf(now) < INFINITY)) ls[r] = 0.0f;
        asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
      }
      const int row0 = tile_row(j);
      const uint32_t at = tmem + t * kCols + lane_base;
      // after a wait that gave up the loop goes on without waiting: every thread
      // still meets the warpgroup's barriers
      if (ok) ok = warp_wait(&sh.s_full[t], (j >> 1) & 1, p.c.err, DERR_FULL_WAIT);
      tc_fence_after();
      if (r == 0) mbar_arrive(&sh.q_empty[j % S::NST]);  // the product has read its queries
      const bool masked = off + row0 < keys + 127 || row0 + kPos > sq.n;
      const int lo = (key - off - row0) * G, hi = (sq.n - row0) * G;
      uint32_t v[2][32];
      uint64_t acc[2] = {0, 0};
      if (odd) {
        // as below, one piece after another, with the scores of the odd columns set
#pragma unroll 1
        for (int k = 0; k < kCols / 32; ++k) {
          tmem_ld32(at + 32 * k, v[0]);
          tmem_wait_ld();
          tmem_pin<32>(v[0]);
          const uint2 m = sh.odd[t][k];
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float e[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int n = 32 * k + i + w;
              float x = __uint_as_float(v[0][i + w]);
              if (m.y >> (i + w) & 1) x = NAN;
              if (n < lo || n >= hi || (m.x >> (i + w) & 1)) x = -INFINITY;
              e[w] = ex2(fmaf(x, ex.c, ls[n]));
            }
            acc[0] = add2(acc[0], pack2(e[0], e[1]));
            acc[1] = add2(acc[1], pack2(e[2], e[3]));
          }
        }
        tc_fence_before();
        mbar_arrive(&sh.s_free[t]);
      } else {
        // 32 columns at a time, the next ones on their way
        tmem_ld32(at, v[0]);
#pragma unroll
        for (int k = 0; k < kCols / 32; ++k) {
          tmem_wait_ld();
          tmem_pin<32>(v[k & 1]);
          if (k < kCols / 32 - 1) {
            tmem_ld32(at + 32 * (k + 1), v[(k + 1) & 1]);
          } else {
            tc_fence_before();
            mbar_arrive(&sh.s_free[t]);
          }
          uint32_t* x = v[k & 1];
          if (masked) {  // rows before the key, rows of no one: -inf
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * k + i < lo || 32 * k + i >= hi) x[i] = 0xff800000u;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(ls + 32 * k + i);
            const float2 y = unpack2(fma2(pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, pack2(l4.x, l4.y)));
            const float2 z = unpack2(fma2(pack2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), c2, pack2(l4.z, l4.w)));
            acc[0] = add2(acc[0], pack2(ex2(y.x), ex2(y.y)));
            acc[1] = add2(acc[1], pack2(ex2(z.x), ex2(z.y)));
          }
        }
      }
      const float2 a = unpack2(add2(acc[0], acc[1]));
      const float y = (a.x + a.y) - comp, u = sum + y;  // compensated sum over the tiles
      comp = (u - sum) - y;
      sum = u;
    }
    sh.sum[t][r] = sum;
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kTma + 1) {
    tc_fence_after();
    tmem_free(tmem, kBuf * kCols);
  }
  if (SPLIT) cg::this_cluster().sync();
  if (split == 0 && tid < nh * 128 && key0 + tid < sq.ctx) {
    const int h = tid >> 7, r = tid & 127;
    float w = sh.sum[h][r] + sh.sum[2 + h][r];
    if (SPLIT)
      for (int k = 1; k < nsplit; ++k) {
        const Shared* o = cg::this_cluster().map_shared_rank(&sh, k);
        w += o->sum[h][r] + o->sum[2 + h][r];
      }
    bool ok;
    const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, key0 + tid, nullptr, &ok);
    if (ok) atomicAdd(p.c.weights + ((size_t)b * p.c.n_kv_heads + g) * 16 + (tid & 15), w);
  }
  if (SPLIT) cg::this_cluster().sync();  // nobody leaves while its sums are read
}

template <int HD, int G>
cudaError_t launch_t(const PromptParams& p, cudaStream_t st) {
  using S = Shape<HD>;
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_prompt_weights<HD, G, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_prompt_weights<HD, G, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Maps maps;
  const uint64_t qd[3] = {(uint64_t)HD, (uint64_t)p.n_heads, (uint64_t)p.total_q};
  const uint64_t qs[2] = {(uint64_t)HD * 2, (uint64_t)p.q_stride * 2};
  const uint32_t qb[3] = {64, (uint32_t)G, kCols / (uint32_t)G};
  const uint64_t cd[2] = {(uint64_t)HD, (uint64_t)p.c.n_blocks * p.c.n_kv_heads * 16}, cs[1] = {(uint64_t)HD * 2};
  const uint32_t cb[2] = {64, 16};
  if (!encode_tensor_map(&maps.q, false, 3, p.q, qd, qs, qb) || !encode_tensor_map(&maps.k, false, 2, p.c.k, cd, cs, cb))
    return cudaErrorInvalidValue;
  const Exponent ex = make_exponent(HD);
  // Two key tiles per CTA, or one as long as there is an SM for each; clusters where
  // SMs are left.  512 tokens of 32/8 heads, hd 64: 7.8 us with one tile, 9.3 with
  // two; 8 sequences of 4096 with 64/8 heads, hd 128: 1135 with one, 908 with two.
  auto units_of = [&](int tiles) {
    return (int64_t)((p.c.max_ctx + 128 * tiles - 1) / (128 * tiles)) * p.n_seqs * p.c.n_kv_heads;
  };
  const int key_tiles = units_of(1) <= sms ? 1 : kTiles;
  const int64_t units = units_of(key_tiles);
  int split = 1;
  while (split < kMaxCluster && units * split * 2 <= sms) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  if (split == 1) return cudaLaunchKernelEx(&cfg, k_prompt_weights<HD, G, false>, p, maps, ex, key_tiles);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_prompt_weights<HD, G, true>, p, maps, ex, key_tiles);
}

}  // namespace

cudaError_t launch_prompt_weights(const PromptParams& p, cudaStream_t st) {
  const int G = p.n_heads / p.c.n_kv_heads, hd = p.c.head_dim;
#define EE_WEIGHTS_CASE(HD_, G_) \
  if (hd == HD_ && G == G_) return launch_t<HD_, G_>(p, st);
  EE_WEIGHTS_CASE(64, 1)
  EE_WEIGHTS_CASE(64, 2)
  EE_WEIGHTS_CASE(64, 4)
  EE_WEIGHTS_CASE(64, 8)
  EE_WEIGHTS_CASE(128, 1)
  EE_WEIGHTS_CASE(128, 2)
  EE_WEIGHTS_CASE(128, 4)
  EE_WEIGHTS_CASE(128, 8)
#undef EE_WEIGHTS_CASE
  return cudaErrorInvalidValue;
}

}  // namespace ee
