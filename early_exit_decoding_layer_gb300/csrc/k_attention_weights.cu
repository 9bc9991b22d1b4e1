// Decode attention over the paged cache that also adds what each token weighs.
//
// A cluster of C CTAs serves one (sequence, kv head) and all query heads of its
// group from one read of K and V; rank r takes a contiguous share of the 16-slot
// blocks, its warps take blocks in turn.  Every warp runs a pipeline of its
// own: K and V of a block come by TMA (128-byte swizzle) into the warp's
// ring, so no warp waits for another until the end.
//  * scores: lane = (token of the block, half of the head's dims), so the sum over
//    the dims stays in the lane but for one exchange between the halves; the
//    swizzle spreads the 16 rows over the banks;
//  * softmax: a running maximum per head and warp that may lag by 2^8, so that
//    rescaling is rare, and a sum per lane;
//  * output: lane = dims, all 16 tokens in turn, probabilities from shared memory.
// The scores stay in shared memory (fp32, every token of the CTA's share).  At the
// end the warps and then, through distributed shared memory, the CTAs join
// (m, l, acc) in a fixed order; with the final m and l known everywhere each CTA
// turns its own scores into weights.  One launch, no scratch, K and V read once;
// everything is fp32 but the fp16 cache.
#include <cooperative_groups.h>
#include <math.h>
#include <stdlib.h>

#include <atomic>

#include "ee_cache_ops.cuh"
#include "ee_tcgen05.cuh"

namespace cg = cooperative_groups;

namespace ee {
namespace {

constexpr int kWarps = 6;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;  // blocks of a warp in shared memory
constexpr int kMaxCluster = 16;

struct Maps {
  CUtensorMap k, v;
};

template <int HD, int G>
struct Layout {
  static constexpr uint32_t kTile = 16 * HD * 2;  // K or V of one block and kv head
  static constexpr uint32_t kRing = kWarps * kStages * 2 * kTile;
  // what is joined, in the ring's space: acc [warp][G][HD], then the CTA's [G][HD]
  static_assert((kWarps + 1) * G * HD * 4 <= kRing, "join space");
};

template <int HD, int G>
struct Shared {
  uint64_t full[kWarps][kStages];
  alignas(16) float q[G][HD];
  alignas(16) float p[kWarps][16][G];
  float wm[kWarps][G], wl[kWarps][G];
  float m[G], l[G];                      // of the CTA
  float cm[kMaxCluster][G], cl[kMaxCluster][G];  // of every rank
  float f[kMaxCluster][G];               // what a rank's acc counts in the whole
  float M[G], inv[G];                    // of the whole sequence
};

template <int HD, int G>
__global__ void __launch_bounds__(kThreads)
    k_attention_weights(const DecodeWeightsParams p, const __grid_constant__ Maps maps, const float c) {
  using Lay = Layout<HD, G>;
  constexpr int E = HD / 32;  // output dims per lane
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<HD, G> sh;
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x / C, g = unit % p.c.n_kv_heads, s = unit / p.c.n_kv_heads;
  const int at = p.pos[s];
  const int n = checked_length(at == INT32_MAX ? at : at + 1, p.c.max_ctx, p.c.err);
  const int nb = (n + 15) >> 4, each = (nb + C - 1) / C;
  const int b0 = min(nb, rank * each), b1 = min(nb, b0 + each);
  const int cap = ((p.c.max_ctx + 15) / 16 + C - 1) / C * 16;  // tokens of a CTA's share at most
  float* sc = reinterpret_cast<float*>(ring + Lay::kRing);     // [G][cap], scores in log2 units
  const int32_t* bt = p.c.table + (int64_t)s * p.c.table_stride;

  if (tid < kWarps * kStages) {
    mbar_init(&sh.full[tid / kStages][tid % kStages], 1);
    fence_mbar_init();
  }
  const float* qg = p.q + ((size_t)s * p.n_heads + g * G) * HD;
  for (int i = tid; i < G * HD; i += kThreads) sh.q[i / HD][i % HD] = qg[i] * c;
  __syncthreads();

  // this warp's blocks: b0 + warp + kWarps * i, i < mine
  const int mine = max(0, (b1 - b0 - warp + kWarps - 1) / kWarps);
  uint8_t* wring = ring + warp * kStages * 2 * Lay::kTile;
  int ids = 0;  // lane i: block id of this warp's block (base + i)
  auto load_ids = [&](int base) {
    const int i = base + lane;
    ids = i < mine ? bt[b0 + warp + kWarps * i] : 0;
    if (ids < 0 || ids >= p.c.n_blocks) {
      report(p.c.err, EE_DERR_BLOCK);
      ids = 0;
    }
  };
  auto fetch = [&](int i) {  // block i of this warp into its stage; ids cover it
    const int row = (__shfl_sync(0xffffffffu, ids, i & 31) * p.c.n_kv_heads + g) * 16;
    const int st = i % kStages;
    if (lane == 0) mbar_arrive_expect_tx(&sh.full[warp][st], 2 * Lay::kTile);
    __syncwarp();
    if (lane < 2 * (HD / 64)) {
      const int half = lane % (HD / 64), kv = lane / (HD / 64);
      tma_load_2d(smem_addr(wring + (st * 2 + kv) * Lay::kTile + half * 2048), kv ? &maps.v : &maps.k, half * 64, row,
                  &sh.full[warp][st]);
    }
  };
  load_ids(0);
  for (int i = 0; i < min(mine, kStages - 1); ++i) fetch(i);

  float m[G], l[G], acc[G][E];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[h][e] = 0.0f;
  }
  const int tok = lane & 15, hf = lane >> 4;
  bool ok = true;
  for (int i = 0; i < mine; ++i) {
    const int ahead = i + kStages - 1;
    if (ahead < mine) {
      if ((ahead & 31) == 0) load_ids(ahead);
      fetch(ahead);
    }
    const int st = i % kStages;
    if (ok) ok = warp_wait(&sh.full[warp][st], (i / kStages) & 1, p.c.err, DERR_FULL_WAIT);
    const uint8_t* kt = wring + st * 2 * Lay::kTile;
    const uint8_t* vt = kt + Lay::kTile;
    const int b = b0 + warp + kWarps * i, nv = min(16, n - b * 16);
    // (1) scores of token tok, this lane's half of the dims
    float z[G];
#pragma unroll
    for (int h = 0; h < G; ++h) z[h] = 0.0f;
    constexpr int J = HD / 16;  // 8-dim chunks per lane
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int jj = HD == 128 ? j : hf * J + j;
      const uint4 kv = *reinterpret_cast<const uint4*>(kt + (HD == 128 ? hf * 2048 : 0) + sw128(tok, jj));
      float kf[8];
      const uint32_t w[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[u]));
        kf[2 * u] = f.x;
        kf[2 * u + 1] = f.y;
      }
      const int d = hf * (HD / 2) + j * 8;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float4 qa = *reinterpret_cast<const float4*>(&sh.q[h][d]), qb = *reinterpret_cast<const float4*>(&sh.q[h][d + 4]);
        z[h] = fmaf(qa.x, kf[0], z[h]);
        z[h] = fmaf(qa.y, kf[1], z[h]);
        z[h] = fmaf(qa.z, kf[2], z[h]);
        z[h] = fmaf(qa.w, kf[3], z[h]);
        z[h] = fmaf(qb.x, kf[4], z[h]);
        z[h] = fmaf(qb.y, kf[5], z[h]);
        z[h] = fmaf(qb.z, kf[6], z[h]);
        z[h] = fmaf(qb.w, kf[7], z[h]);
      }
    }
    bool grow = false;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      z[h] += __shfl_xor_sync(0xffffffffu, z[h], 16);
      if (tok >= nv) z[h] = -INFINITY;
      grow |= z[h] - m[h] > 8.0f;
    }
    if (__any_sync(0xffffffffu, grow)) {  // the first block, and rarely later
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float mn = fmaxf(m[h], warp_max(z[h]));
        const float a = m[h] == mn ? 1.0f : ex2(m[h] - mn);
        m[h] = mn;
        l[h] *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[h][e] *= a;
      }
    }
    // (2) probabilities, scores kept
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float e = ex2(z[h] - (m[h] == -INFINITY ? 0.0f : m[h]));
      if (hf == 0) {
        l[h] += e;
        sh.p[warp][tok][h] = e;
        sc[h * cap + (b - b0) * 16 + tok] = z[h];
      }
    }
    __syncwarp();
    // (3) output dims of this lane: hd 128: 4 at half lane / 16; hd 64: 2
    auto add = [&](int r) {
      float vf[E];
      if constexpr (HD == 128) {
        const uint2 x = *reinterpret_cast<const uint2*>(vt + hf * 2048 + sw128(r, tok >> 1) + (tok & 1) * 8);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&x.x));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&x.y));
        vf[0] = f0.x, vf[1] = f0.y, vf[2] = f1.x, vf[3] = f1.y;
      } else {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(vt + sw128(r, lane >> 2) + (lane & 3) * 4);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&x));
        vf[0] = f0.x, vf[1] = f0.y;
      }
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float pr = sh.p[warp][r][h];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[h][e] = fmaf(pr, vf[e], acc[h][e]);
      }
    };
    if (nv == 16) {
#pragma unroll
      for (int r = 0; r < 16; ++r) add(r);
    } else {
      for (int r = 0; r < nv; ++r) add(r);  // slots behind the last token may hold anything
    }
    __syncwarp();  // the stage and p are free
  }
  // copies of a wait that gave up land before the space is used again
  if (!ok)
    for (int i = max(0, mine - kStages); i < mine; ++i)
      mbar_wait_bounded(&sh.full[warp][i % kStages], (i / kStages) & 1, p.c.err, DERR_DRAIN_WAIT);

  // the warps join
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float t = warp_sum(l[h]);
    if (lane == 0) {
      sh.wm[warp][h] = m[h];
      sh.wl[warp][h] = t;
    }
  }
  __syncthreads();  // all rings are free
  float* wacc = reinterpret_cast<float*>(ring);  // [warp][G][HD]
  const int d0 = HD == 128 ? hf * 64 + tok * 4 : lane * 2;
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int e = 0; e < E; ++e) wacc[(warp * G + h) * HD + d0 + e] = acc[h][e];
  __syncthreads();
  float* cacc = wacc + kWarps * G * HD;
  for (int i = tid; i < G * HD; i += kThreads) {
    const int h = i / HD;
    float mm = -INFINITY, a = 0.0f, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sh.wm[w][h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = sh.wm[w][h] == mm ? 1.0f : ex2(sh.wm[w][h] - mm);
      if (sh.wl[w][h] != 0.0f) {
        a = fmaf(f, wacc[w * G * HD + i], a);
        ll = fmaf(f, sh.wl[w][h], ll);
      }
    }
    cacc[i] = a;
    if (i % HD == 0) {
      sh.m[h] = mm;
      sh.l[h] = ll;
    }
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
    for (int k = 0; k < kMaxCluster; ++k) v[k] = k < C ? cl.map_shared_rank(cacc, k)[i] : 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < C && sh.f[k][h] != 0.0f) a = fmaf(sh.f[k][h], v[k], a);
    p.o[((size_t)s * p.n_heads + g * G) * HD + i] = a * sh.inv[h];
  }
  // the weights of this CTA's tokens
  for (int t = tid; t < min(n, b1 * 16) - b0 * 16; t += kThreads) {
    float w = 0.0f;
#pragma unroll
    for (int h = 0; h < G; ++h) w = fmaf(ex2(sc[h * cap + t] - sh.M[h]), sh.inv[h], w);
    bool bok;
    const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, b0 * 16 + t, nullptr, &bok);
    if (bok) atomicAdd(p.c.weights + ((size_t)b * p.c.n_kv_heads + g) * 16 + (t & 15), w);
  }
  cl.sync();  // nobody leaves while its part is read
}

template <int HD, int G>
cudaError_t launch_t(const DecodeWeightsParams& p, cudaStream_t st) {
  using Lay = Layout<HD, G>;
  constexpr int kMaxSmem = 227 * 1024 - (int)sizeof(Shared<HD, G>) - 1024;
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_attention_weights<HD, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_attention_weights<HD, G>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Maps maps;
  const uint64_t cd[2] = {(uint64_t)HD, (uint64_t)p.c.n_blocks * p.c.n_kv_heads * 16}, cs[1] = {(uint64_t)HD * 2};
  const uint32_t cb[2] = {64, 16};
  if (!encode_tensor_map(&maps.k, false, 2, p.c.k, cd, cs, cb) || !encode_tensor_map(&maps.v, false, 2, p.c.v, cd, cs, cb))
    return cudaErrorInvalidValue;
  // enough CTAs for two per SM, shares of at least one block per warp, and the scores of
  // a share in shared memory
  const int units = p.batch * p.c.n_kv_heads, nb = (p.c.max_ctx + 15) / 16;
  auto smem = [&](int C) { return 1024 + (size_t)Lay::kRing + (size_t)G * ((nb + C - 1) / C) * 16 * 4; };
  int C = 1;
  const char* ec = getenv("EE_C");
  if (ec) C = atoi(ec); else
  while (C < kMaxCluster && (smem(C) > (size_t)kMaxSmem || (units * C < 2 * sms && nb > C * kWarps))) C *= 2;
  if (smem(C) > (size_t)kMaxSmem) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem(C);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attention_weights<HD, G>, p, maps,
                            (float)(1.4426950408889634074 / sqrt((double)HD)));
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
