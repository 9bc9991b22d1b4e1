// Eviction from the paged cache by accumulated weight.
//
// A cluster of C CTAs serves one (sequence, kv head).  Every CTA finds the kept
// tokens for itself (a few microseconds; sharing that work would cost a cluster
// barrier per step), and the CTAs share the moving of the rows, which is what the
// bytes are.
//
// Selection: the keep - recent heaviest of the tokens before the last `recent`, by
// radix selection on the weights' bits, mapped to unsigned integers of the same
// order: four passes of 8 bits, each a histogram, its suffix sums and the digit in
// which the wanted rank falls.  Accumulated weights are of similar size, so
// most keys fall into a few bins of the first pass: the histogram has a
// copy per lane, which keeps the lanes of a warp off each other's counters.
// Tokens above the resulting key stay, and of those equal to it the first ones, so
// ties go to the lower index.  Each thread owns a run of tokens, so two prefix sums
// (equal ones, then kept ones) give every kept token its slot.
//
// Moving: a kept token's slot is never above the token, so rows move in place in
// ascending order: the cluster reads a chunk of rows into registers (K, V and
// weight), meets, and writes it; later chunks read only rows behind it.  Into
// other blocks nothing has to meet.
#include <cooperative_groups.h>
#include <math.h>

#include <atomic>

#include "ee_cache_ops.cuh"

namespace cg = cooperative_groups;

namespace ee {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kPieces = 4;  // 16-byte pieces of K, and of V, in a thread's registers

// Unsigned integers in the order of the floats, -0 as 0 and NaN below all.
EE_DEV uint32_t order_key(float f) {
  if (isnan(f)) return 0u;
  const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of one value per thread.
EE_DEV int block_scan(int v, int* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warps is free again
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) base += warps[w];
  return base + x - v;
}

// A thread's run of tokens lies apart from the next one's by an odd number of words.
EE_DEV int pad(int t) { return t + (t >> 5); }

// Shared memory: keys (padded), then the histograms; the kept tokens (16 bits: below
// 2^14) over the histograms; the two block tables.
struct Layout {
  int keys, kept, src, dst, bytes;
};
__host__ __device__ inline Layout layout(int max_ctx, int keep) {
  Layout l;
  l.keys = 0;
  l.kept = (max_ctx + max_ctx / 32 + 1) * 4;
  l.kept = (l.kept + 15) / 16 * 16;
  const int hist = 256 * 32 * 4, list = (max_ctx * 2 + 15) / 16 * 16;
  l.src = l.kept + (hist > list ? hist : list);
  l.dst = l.src + (max_ctx + 15) / 16 * 4;
  l.bytes = l.dst + (keep + 15) / 16 * 4;
  return l;
}

template <int HD>
__global__ void __launch_bounds__(kThreads) k_evict(const EvictParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int warps[kWarps], s_digit, s_above;
  __shared__ int bins[256];
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, hkv = p.c.n_kv_heads;
  const int unit = blockIdx.x / C, g = unit % hkv, s = unit / hkv;
  const Layout lay = layout(p.c.max_ctx, p.keep);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + lay.keys);
  int* hist = reinterpret_cast<int*>(smem + lay.kept);
  uint16_t* kept = reinterpret_cast<uint16_t*>(smem + lay.kept);
  int* src = reinterpret_cast<int*>(smem + lay.src);
  int* dst = reinterpret_cast<int*>(smem + lay.dst);
  const int n = checked_length(p.ctx[s], p.c.max_ctx, p.c.err);
  const int len = min(n, p.keep);
  const bool in_place = p.dst_table == p.c.table;
  if (g == 0 && rank == 0 && tid == 0) p.new_ctx[s] = len;

  // block ids, -1 where out of range
  auto load_table = [&](const int32_t* table, int64_t stride, int blocks, int* to) {
    for (int b = tid; b < blocks; b += kThreads) {
      int id = table[s * stride + b];
      if (id < 0 || id >= p.c.n_blocks) {
        report(p.c.err, EE_DERR_BLOCK);
        id = -1;
      }
      to[b] = id;
    }
  };
  load_table(p.c.table, p.c.table_stride, (n + 15) >> 4, src);
  load_table(p.dst_table, p.dst_stride, (len + 15) >> 4, dst);
  __syncthreads();

  if (n <= p.keep) {
    for (int i = tid; i < n; i += kThreads) kept[i] = (uint16_t)i;
  } else {
    const int m = n - p.recent;          // candidates
    const int need = p.keep - p.recent;  // of them, fewer than m
    for (int i = tid; i < (m + 3) / 4; i += kThreads) {
      const float4 w = *reinterpret_cast<const float4*>(p.c.weights + ((size_t)max(src[i >> 2], 0) * hkv + g) * 16 + (i & 3) * 4);
      const float f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (4 * i + u < m) keys[pad(4 * i + u)] = order_key(f[u]);
    }
    uint32_t prefix = 0, mask = 0;
    int rest = need;  // rank of the key looked for, among those that match the prefix
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
      for (int i = tid; i < 256 * 32; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int t = tid; t < m; t += kThreads) {
        const uint32_t k = keys[pad(t)];
        if ((k & mask) == prefix) atomicAdd(&hist[((k >> shift) & 255) * 32 + lane], 1);
      }
      __syncthreads();
      for (int b = tid >> 5; b < 256; b += kWarps) {
        const int c = (int)__reduce_add_sync(0xffffffffu, (unsigned)hist[b * 32 + lane]);
        if (lane == 0) bins[b] = c;
      }
      __syncthreads();
      if (tid < 32) {  // lane l: bins 8 l .. 8 l + 7, from the top
        int c[8], sum = 0;
#pragma unroll
        for (int u = 7; u >= 0; --u) sum += (c[u] = bins[(31 - lane) * 8 + u]);
        int above = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, above, o);
          if (lane >= o) above += y;
        }
        above -= sum;  // keys in higher lanes' bins
        if (above < rest && above + sum >= rest) {
#pragma unroll
          for (int u = 7; u >= 0; --u) {
            if (above < rest && above + c[u] >= rest) {
              s_digit = (31 - lane) * 8 + u;
              s_above = above;
            }
            above += c[u];
          }
        }
      }
      __syncthreads();
      rest -= s_above;
      prefix |= (uint32_t)s_digit << shift;
      mask |= 255u << shift;
    }
    // tokens [t0, t1) are this thread's; keys above prefix stay, and the first `rest`
    // equal ones, and the recent tokens
    const int each = (n + kThreads - 1) / kThreads;
    const int t0 = min(n, tid * each), t1 = min(n, t0 + each);
    int equal = 0, more = 0;
    for (int t = t0; t < t1; ++t) {
      const bool cand = t < m && need > 0;
      const uint32_t k = cand ? keys[pad(t)] : 0u;
      equal += cand && k == prefix;
      more += t >= m || (cand && k > prefix);
    }
    const int before = block_scan(equal, warps);
    const int ties = max(0, min(equal, rest - before));
    int slot = block_scan(more + ties, warps);
    int taken = 0;
    for (int t = t0; t < t1; ++t) {  // the histograms are no longer read
      const bool cand = t < m && need > 0;
      const uint32_t k = cand ? keys[pad(t)] : 0u;
      bool stay = t >= m || (cand && k > prefix);
      if (cand && k == prefix && taken < ties) {
        stay = true;
        ++taken;
      }
      if (stay) kept[slot++] = (uint16_t)t;
    }
  }
  __syncthreads();
  if (p.kept)
    for (int i = rank * kThreads + tid; i < p.keep; i += C * kThreads)
      p.kept[((size_t)s * hkv + g) * p.keep + i] = i < len ? kept[i] : -1;
  if (n <= p.keep && in_place) return;  // nothing moves, in the whole cluster

  constexpr int P = HD / 8;                       // pieces per row
  constexpr int kChunk = kThreads * kPieces / P;  // rows per CTA and step
  uint4* kc = reinterpret_cast<uint4*>(const_cast<uint16_t*>(p.c.k));
  uint4* vc = reinterpret_cast<uint4*>(const_cast<uint16_t*>(p.c.v));
  const int j = tid % P;
  for (int step = 0; step < len; step += C * kChunk) {
    uint4 a[kPieces], b[kPieces];
    float w[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = step + rank * kChunk + u * (kThreads / P) + tid / P;
      const int t = i < len ? kept[i] : 0;
      if (i < len && !(in_place && t == i)) {
        const size_t at = ((size_t)max(src[t >> 4], 0) * hkv + g) * 16 + (t & 15);
        a[u] = kc[at * P + j];
        b[u] = vc[at * P + j];
        if (j == 0) w[u] = p.c.weights[at];
      }
    }
    if (in_place) cl.sync();
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = step + rank * kChunk + u * (kThreads / P) + tid / P;
      if (i < len && !(in_place && kept[i] == i) && dst[i >> 4] >= 0) {
        const size_t at = ((size_t)dst[i >> 4] * hkv + g) * 16 + (i & 15);
        kc[at * P + j] = a[u];
        vc[at * P + j] = b[u];
        if (j == 0) p.c.weights[at] = w[u];
      }
    }
  }
}

template <int HD>
cudaError_t launch_t(const EvictParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_evict<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             layout(kCacheMaxCtx, kCacheMaxCtx).bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_evict<HD>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // CTAs for every SM, as long as each has a chunk of rows to move
  const int units = p.batch * p.c.n_kv_heads, chunk = kThreads * kPieces / (HD / 8);
  int C = 1;
  while (C < kMaxCluster && units * C < sms && C * chunk < p.keep) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = layout(p.c.max_ctx, min(p.keep, p.c.max_ctx)).bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_evict<HD>, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t st) {
  return p.c.head_dim == 64 ? launch_t<64>(p, st) : launch_t<128>(p, st);
}

}  // namespace ee
