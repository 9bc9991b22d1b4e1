// Decode attention over the paged cache that also adds what each token weighs, on
// the tensor cores.
//
// One new token per sequence: K and V are read once for the G query heads of a kv
// head, 2 G products per element, so the bytes are the bound -- if the arithmetic
// keeps out of the way.  On the CUDA cores (a token per lane, fp32 fma) it did not:
// 1100 instructions per 16-slot block and warp held 32 sequences of up to 2176
// tokens at 45 us, where the bytes take 23.  So both products run as MMAs with
// the cache as the big operand:
//   S = K_tile Q^T    64 tokens x 16 columns
//   O^T = V_tile^T P  head dims x 16 columns, K = 64 tokens
// fp32 queries and probabilities go in as fp16 pairs, x = hi + lo, columns h and
// 8 + h: 22 bits, which keeps the fp32 result.  A query head is scaled by a power
// of two to a largest value near 2^10, and probabilities by 2^7, so that neither
// part falls below fp16's range.  Each tile's O is a product of its own, added to
// fp32 registers: the tensor core cuts its accumulator after every step, which
// over 16384 tokens would show.
//
// A cluster of C CTAs serves one (sequence, kv head), each a share of the 16-slot
// blocks, in tiles of four:
//   warps 0-3  a thread per token: scores, a running maximum that may lag by 2^8 (so
//              that rescaling is rare), probabilities into shared memory;
//              then a thread per head dim adds O
//   warp 4     K and V tiles by TMA into a ring
//   warp 5     (one thread) the MMAs, S a tile ahead of O
// The scores of the share stay in shared memory.  At the end the CTAs join (m, l, O)
// through distributed shared memory in rank order, and each turns its own scores
// into weights.  One launch, no scratch, K and V read once.
//
// 32 sequences of 8192 tokens, 32/8 heads, hd 128: 210 us, 5.1 TB/s (0.76 of the
// measured copy rate); 257 to 2176 tokens: 39 us, 4.0 TB/s, where two rounds of CTAs
// with 6 us each of launch, first loads and join show; one of 2113: 8.7 us.
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

constexpr int kThreads = 192;
constexpr int kTokens = 64;  // per tile
constexpr int kMaxCluster = 12;
constexpr float kLift = 7.0f;  // probabilities are 2^kLift times their value

struct Maps {
  CUtensorMap k, v;
};

template <int HD>
struct Layout {
  static constexpr int H = HD / 64;                     // 64-column halves
  static constexpr uint32_t kTile = kTokens * HD * 2;   // K or V of one tile
  static constexpr uint32_t kHalf = kTokens * 128;      // one half of it
  static constexpr int NS = HD == 128 ? 5 : 8;          // ring tiles
  static constexpr uint32_t kQ = H * 2048, kP = 2048;   // 16 rows of 128 bytes each
  static constexpr uint32_t kFixed = NS * kTile + kQ + 2 * kP;
};

template <int HD, int G>
struct Shared {
  uint64_t full[Layout<HD>::NS], empty[Layout<HD>::NS], s_full[2], p_ready[2], o_full[2];
  uint32_t tmem;
  float unscale[8], red[4][8];
  float m[G], l[G];                              // of the CTA
  float cm[kMaxCluster][G], cl[kMaxCluster][G];  // of every rank
  float f[kMaxCluster][G];                       // what a rank's O counts in the whole
  float M[G], inv[G];                            // of the whole sequence
};

// The sequence with the r-th largest position (equal ones by index); a whole warp.
EE_DEV int nth_longest(const int32_t* pos, int batch, int r) {
  static_assert(EE_MAX_BATCH <= 64, "two sequences per lane");
  const int lane = threadIdx.x & 31;
  const int a = lane < batch ? pos[lane] : INT_MIN, b = lane + 32 < batch ? pos[lane + 32] : INT_MIN;
  int ra = 0, rb = 0;  // how many come before
#pragma unroll 4
  for (int k = 0; k < min(batch, 32); ++k) {
    const int x = __shfl_sync(0xffffffffu, a, k), y = __shfl_sync(0xffffffffu, b, k);
    ra += (x > a || (x == a && k < lane)) + (y > a);
    rb += (x >= b) + (y > b || (y == b && k < lane));
  }
  const unsigned ha = __ballot_sync(0xffffffffu, lane < batch && ra == r);
  const unsigned hb = __ballot_sync(0xffffffffu, lane + 32 < batch && rb == r);
  return ha ? __ffs(ha) - 1 : 31 + __ffs(hb);
}

// hi + lo of a value that went in as two fp16 parts.  Where hi is not finite, lo is no
// part of it (0 times infinity).
EE_DEV float whole(uint32_t hi, uint32_t lo) {
  return (hi & 0x7f800000u) == 0x7f800000u ? __uint_as_float(hi) : __uint_as_float(hi) + __uint_as_float(lo);
}

template <int HD, int G>
__global__ void __launch_bounds__(kThreads, 2)
    k_attention_weights(const DecodeWeightsParams p, const __grid_constant__ Maps maps, const float c) {
  using Lay = Layout<HD>;
  constexpr int NS = Lay::NS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<HD, G> sh;
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* qs = ring + NS * Lay::kTile;
  uint8_t* ps = qs + Lay::kQ;
  float* sc = reinterpret_cast<float*>(ring + Lay::kFixed);  // [G][cap], scores in log2 units
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // long sequences first: the grid's last CTAs are then short ones
  const int unit = blockIdx.x / C, g = unit % p.c.n_kv_heads, s = nth_longest(p.pos, p.batch, unit / p.c.n_kv_heads);
  const int at = p.pos[s];
  const int n = checked_length(at == INT32_MAX ? at : at + 1, p.c.max_ctx, p.c.err);
  const int nb = (n + 15) >> 4, each = (nb + C - 1) / C;
  const int b0 = min(nb, rank * each), b1 = min(nb, b0 + each);
  const int nt = (b1 - b0 + 3) >> 2;                        // tiles of this CTA
  const int have = max(0, min(n, b1 * 16) - b0 * 16);       // its tokens
  const int cap = ((p.c.max_ctx + 15) / 16 + C - 1) / C * 16;  // at most
  int* ids = reinterpret_cast<int*>(sc + (size_t)G * cap);     // [cap / 16], its blocks, -1 where out of range

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_ready[i], 128);
      mbar_init(&sh.o_full[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 5) tmem_alloc(&sh.tmem, 64);
  // rows of Q and P without a head are zero
  for (int i = tid; i < (int)(Lay::kQ + 2 * Lay::kP) / 16; i += kThreads)
    reinterpret_cast<uint4*>(qs)[i] = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  auto stage = [&](int i) { return i % NS; };
  auto phase = [&](int i) { return (uint32_t)(i / NS) & 1; };

  if (warp == 4) {
    // ring item 2 j is K of tile j, item 2 j + 1 its V
    const int b4 = lane & 3, half = lane >> 2;
    const int32_t* bt = p.c.table + (int64_t)s * p.c.table_stride + b0;
    auto block_id = [&](int j) {
      const int b = 4 * j + b4;
      int id = b < b1 - b0 ? bt[b] : 0;
      const bool bad = id < 0 || id >= p.c.n_blocks;
      if (bad) {
        report(p.c.err, EE_DERR_BLOCK);
        id = 0;
      }
      if (b < b1 - b0 && half == 0) ids[b] = bad ? -1 : id;
      return id;
    };
    int id = block_id(0), issued = 0;
    bool ok = true;
    for (int j = 0; j < nt && ok; ++j) {
      const int next = block_id(j + 1), here = min(4, b1 - b0 - 4 * j);
      for (int kv = 0; kv < 2; ++kv, ++issued) {
        const int st = stage(issued);
        if (issued >= NS) ok = warp_wait(&sh.empty[st], phase(issued - NS), p.c.err, DERR_EMPTY_WAIT);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], (uint32_t)here * 16 * HD * 2);
        __syncwarp();
        if (half < Lay::H && b4 < here)
          tma_load_2d(smem_addr(ring + st * Lay::kTile + half * Lay::kHalf + b4 * 2048), kv ? &maps.v : &maps.k, half * 64,
                      (id * p.c.n_kv_heads + g) * 16, &sh.full[st]);
      }
      id = next;
    }
    if (!ok)  // copies land before the CTA ends
      for (int i = max(0, issued - NS); i < issued; ++i)
        mbar_wait_bounded(&sh.full[stage(i)], phase(i), p.c.err, DERR_DRAIN_WAIT);
  } else if (warp == 5) {
    asm volatile("bar.sync 2, 160;" ::: "memory");  // Q is in place
    if (lane == 0 && nt > 0) {
      constexpr uint32_t id_s = instr_desc(0, 16, kTokens), id_o = instr_desc(0, 16, HD, false, true);
      const uint64_t qd = smem_desc_sw128(smem_addr(qs));
      auto landed = [&](int i) {
        const bool r = mbar_wait_bounded(&sh.full[stage(i)], phase(i), p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        return r;
      };
      auto scores = [&](int j) {
        const uint64_t k = smem_desc_sw128(smem_addr(ring) + stage(2 * j) * Lay::kTile);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_f16(tmem + (j & 1) * 16, k + (((kk >> 2) * Lay::kHalf + (kk & 3) * 32) >> 4),
                  qd + (((kk >> 2) * 2048 + (kk & 3) * 32) >> 4), id_s, kk > 0);
        mma_commit(&sh.s_full[j & 1]);
      };
      bool ok = landed(0);
      if (ok) scores(0);
#pragma unroll 1
      for (int j = 0; j < nt && ok; ++j) {
        if (j + 1 < nt) {
          if (!(ok = landed(2 * j + 2))) break;
          scores(j + 1);
        }
        if (!(ok = mbar_wait_bounded(&sh.p_ready[j & 1], (j >> 1) & 1, p.c.err, DERR_FULL_WAIT) && landed(2 * j + 1))) break;
        const uint64_t v = smem_desc_sw128_mn(smem_addr(ring) + stage(2 * j + 1) * Lay::kTile, Lay::kHalf);
        const uint64_t pd = smem_desc_sw128(smem_addr(ps) + (j & 1) * Lay::kP);
#pragma unroll
        for (int kk = 0; kk < kTokens / 16; ++kk)
          mma_f16(tmem + 32 + (j & 1) * 16, v + kk * (2048 >> 4), pd + kk * (32 >> 4), id_o, kk > 0);
        mma_commit(&sh.o_full[j & 1]);
      }
    }
    __syncwarp();
  } else {
    // Q: head h = warp, warp + 4
    const float* qg = p.q + ((size_t)s * p.n_heads + g * G) * HD;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = warp + 4 * u;
      if (h < G) {
        float x[HD / 32], big = 0.0f;
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) {
          x[e] = qg[h * HD + e * 32 + lane] * c;
          big = fmaxf(big, fabsf(x[e]));
        }
        big = warp_max(big);
        // 2^k with 2^9 <= big 2^k < 2^10, k within +-60
        int k = 136 - (int)(__float_as_uint(big) >> 23);
        k = max(-60, min(60, k));
        const float up = __uint_as_float((uint32_t)(127 + k) << 23);
        if (lane == 0) sh.unscale[h] = __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) {
          const int d = e * 32 + lane;
          const float y = x[e] * up;
          const __half hi = __float2half_rn(y), lo = __float2half_rn(y - __half2float(hi));
          uint8_t* to = qs + (d >> 6) * 2048 + (d & 7) * 2;
          *reinterpret_cast<__half*>(to + sw128(h, (d & 63) >> 3)) = hi;
          *reinterpret_cast<__half*>(to + sw128(8 + h, (d & 63) >> 3)) = lo;
        }
      }
    }
    fence_proxy_async();
    asm volatile("bar.sync 2, 160;" ::: "memory");
    float unscale[G], m[G], l[G], acc[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      unscale[h] = sh.unscale[h];
      m[h] = -INFINITY;
      l[h] = 0.0f;
      acc[h] = 0.0f;
    }
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    // M = 64: rows 16 w .. 16 w + 15 in the first lanes of warp w's part of tensor memory
    const bool is_token = lane < 16;
    const int tok = warp * 16 + (lane & 15);
    // after a wait that gave up the loop goes on without waiting: every thread
    // still meets the warps' barriers
    bool ok = true;
    auto add_output = [&](int j) {
      if (ok) ok = warp_wait(&sh.o_full[j & 1], (j >> 1) & 1, p.c.err, DERR_FULL_WAIT);
      tc_fence_after();
      if (tid == 0) mbar_arrive(&sh.empty[stage(2 * j + 1)]);
      uint32_t v[16];
      tmem_ld16(tmem + 32 + (j & 1) * 16 + lane_base, v);
      tmem_wait_ld();
      tmem_pin<16>(v);
#pragma unroll
      for (int h = 0; h < G; ++h) acc[h] += whole(v[h], v[8 + h]);
    };
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      if (ok) ok = warp_wait(&sh.s_full[j & 1], (j >> 1) & 1, p.c.err, DERR_FULL_WAIT);
      tc_fence_after();
      if (tid == 0) mbar_arrive(&sh.empty[stage(2 * j)]);
      uint32_t v[16];
      tmem_ld16(tmem + (j & 1) * 16 + lane_base, v);
      tmem_wait_ld();
      tmem_pin<16>(v);
      const int left = have - j * kTokens;  // tokens from this tile on
      const bool live = is_token && tok < left;
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
      uint8_t* pt = ps + (j & 1) * Lay::kP + (tok & 7) * 2;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float e = ex2(z[h] - (m[h] == -INFINITY ? 0.0f : m[h]) + kLift);
        l[h] += e;
        if (is_token) {
          const __half hi = __float2half_rn(e), lo = __float2half_rn(e - __half2float(hi));
          *reinterpret_cast<__half*>(pt + sw128(h, tok >> 3)) = hi;
          *reinterpret_cast<__half*>(pt + sw128(8 + h, tok >> 3)) = lo;
        }
        if (live) sc[h * cap + j * kTokens + tok] = z[h];
      }
      if (left < kTokens) {
        // slots behind the last token hold anything: their V becomes zero
        if (ok) ok = warp_wait(&sh.full[stage(2 * j + 1)], phase(2 * j + 1), p.c.err, DERR_FULL_WAIT);
        const int r = tid & 63, half = tid >> 6;
        if (r >= left && half < Lay::H) {
          uint4* row = reinterpret_cast<uint4*>(ring + stage(2 * j + 1) * Lay::kTile + half * Lay::kHalf + r * 128);
#pragma unroll
          for (int k = 0; k < 8; ++k) row[k] = make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&sh.p_ready[j & 1]);
      if (j > 0) add_output(j - 1);
#pragma unroll
      for (int h = 0; h < G; ++h) acc[h] *= a[h];
    }
    if (nt > 0) add_output(nt - 1);
    // this CTA's (m, l, O); the ring is free
    float* cacc = reinterpret_cast<float*>(ring);  // [G][HD]
    const int dim = HD == 128 ? tid : tok;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float t = warp_sum(l[h]);
      if (lane == 0) sh.red[warp][h] = t;
      if (HD == 128 || is_token) cacc[h * HD + dim] = acc[h];
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (tid < G) sh.l[tid] = (sh.red[0][tid] + sh.red[1][tid]) + (sh.red[2][tid] + sh.red[3][tid]);
    if (tid == 0)
#pragma unroll
      for (int h = 0; h < G; ++h) sh.m[h] = m[h];
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_free(tmem, 64);
  }
  cl.sync();
  // the CTAs join: every rank finds M and L, rank r a share of the outputs
  for (int i = tid; i < C * G; i += kThreads) {
    const Shared<HD, G>* o = cl.map_shared_rank(&sh, i / G);
    sh.cm[i / G][i % G] = o->m[i % G];
    sh.cl[i / G][i % G] = o->l[i % G];
  }
  __syncthreads();
  if (tid < G) {
    float mm = -INFINITY, ll = 0.0f;
    for (int k = 0; k < C; ++k) mm = fmaxf(mm, sh.cm[k][tid]);
    for (int k = 0; k < C; ++k) {
      const float f = sh.cl[k][tid] == 0.0f ? 0.0f : sh.cm[k][tid] == mm ? 1.0f : ex2(sh.cm[k][tid] - mm);
      sh.f[k][tid] = f;
      if (f != 0.0f) ll = fmaf(f, sh.cl[k][tid], ll);
    }
    sh.M[tid] = mm;
    sh.inv[tid] = ll == 0.0f ? 0.0f : 1.0f / ll;
  }
  __syncthreads();
  const int share = (G * HD + C - 1) / C;
  for (int i = rank * share + tid; i < min(G * HD, (rank + 1) * share); i += kThreads) {
    const int h = i / HD;
    float v[kMaxCluster], a = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) v[k] = k < C ? cl.map_shared_rank(reinterpret_cast<float*>(ring), k)[i] : 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < C && sh.f[k][h] != 0.0f) a = fmaf(sh.f[k][h], v[k], a);
    p.o[((size_t)s * p.n_heads + g * G) * HD + i] = a * sh.inv[h];
  }
  // the weights of this CTA's tokens; inv has the probabilities' 2^kLift
  for (int t = tid; t < have; t += kThreads) {
    float w = 0.0f;
#pragma unroll
    for (int h = 0; h < G; ++h) w = fmaf(ex2(sc[h * cap + t] - sh.M[h] + kLift), sh.inv[h], w);
    const int b = ids[t >> 4];
    if (b >= 0) atomicAdd(p.c.weights + ((size_t)b * p.c.n_kv_heads + g) * 16 + (t & 15), w);
  }
  cl.sync();  // nobody leaves while its part is read
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
  const uint64_t cd[2] = {(uint64_t)HD, (uint64_t)p.c.n_blocks * p.c.n_kv_heads * 16}, cs[1] = {(uint64_t)HD * 2};
  const uint32_t cb[2] = {64, 16};
  if (!encode_tensor_map(&maps.k, false, 2, p.c.k, cd, cs, cb) || !encode_tensor_map(&maps.v, false, 2, p.c.v, cd, cs, cb))
    return cudaErrorInvalidValue;
  // The cluster size with the least estimated time: waves of CTAs, each a fixed part
  // (launch, first loads, join: 6 us measured) and its tiles, which take 0.87 us one
  // after another, or their bytes at an SM's share of the memory's bandwidth (44.5
  // GB/s) times the CTAs that share it.  The scores of a share decide how many CTAs
  // an SM holds, the GPCs (of up to 20 SMs) how many clusters fit.  Estimated
  // and measured, 8 kv heads of 128, 4 query heads each: 32 sequences of 2176
  // tokens with C = 1, 2, 3, 4: 71, 62, 66, 74 and 78, 59, 68, 74 us; 8 of 16384
  // with 2, 4, 6, 9, 12: 117, 123, 130, 156, 106 and 126, 129, 136, 163, 102; one of
  // 2113 with 1, 4, 8, 12: 36, 14, 10, 9 and 36, 13.8, 10.5, 8.7.
  const int units = p.batch * p.c.n_kv_heads, nb = (p.c.max_ctx + 15) / 16;
  auto smem = [&](int C) { return 1024 + (size_t)Lay::kFixed + ((nb + C - 1) / C) * (size_t)(G * 16 + 1) * 4; };
  int C = 0;
  double least = 0.0;
  for (int k = 1; k <= kMaxCluster; ++k) {
    const int one = held[dev][k].load(std::memory_order_relaxed);
    if (one < 1 || smem(k) > (size_t)kMaxSmem || (C > 0 && nb <= 4 * (k - 1))) continue;
    const int fit = std::max<int>(1, std::min<int>(4, 228 * 1024 / (int)(smem(k) + sizeof(Shared<HD, G>) + 1024)));
    const int ctas = units * k, slots = one * fit, waves = (ctas + slots - 1) / slots;
    const double live = (double)std::min(ctas, slots) / sms;
    const int tiles = ((nb + k - 1) / k + 3) / 4;
    const double t = waves * (6.0 + tiles * std::max(0.87, live * (2.0 * Lay::kTile / 44.5e3)));
    if (C == 0 || t < least) {
      C = k;
      least = t;
    }
  }
  if (C == 0) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.dynamicSmemBytes = smem(C);
  cfg.stream = st;
  attr[0].val.clusterDim.x = C;
  return cudaLaunchKernelEx(&cfg, k_attention_weights<HD, G>, p, maps, make_exponent(HD).c);
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
