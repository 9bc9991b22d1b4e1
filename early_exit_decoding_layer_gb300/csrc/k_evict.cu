// Eviction from the paged cache by accumulated weight.
//
// A cluster of C CTAs serves one (sequence, kv head).  Every CTA finds the kept
// tokens for itself (a few microseconds; sharing that work would cost a cluster
// barrier per step), and the CTAs share the moving of the rows, which is what the
// bytes are.
//
// Selection: the keep - recent heaviest of the tokens before the last `recent`, by
// radix selection on the weights' bits, mapped to unsigned integers of the same
// order: up to four passes of 8 bits, each a histogram, its sums from the top and
// the digit in which the wanted rank falls; a digit whose keys all stay ends
// it.  Accumulated weights are of similar size, so most keys fall into a few bins
// of the first pass: the histogram has eight copies, which leaves four lanes of a
// warp on a counter (32 copies: clearing and adding them cost 2600 cycles a
// pass, with 500 keys as with 16000).  Tokens above the resulting key stay, and of
// those equal to it the first ones, so ties go to the lower index.  Warps own runs
// of tokens, of which lane i keeps the i-th 32 as a word of bits: slots come from
// one scan over the words (with ballots and a running slot per 32 tokens, in
// two walks, this took 10200 cycles of 35000 at 16384 tokens, now 4600).
//
// Moving: a kept token's slot is never above the token, so rows move in place in
// ascending order: the cluster reads a chunk of rows into registers (K, V and
// weight), meets, and writes it; later chunks read only rows behind it.  Into
// other blocks nothing has to meet.
//
// Bound: kept rows read and written.  32 sequences of 256 to 2304 tokens cut to
// 1024, 8 kv heads, hd 128: 48 us, 5.4 TB/s (0.80 of the measured copy rate); one of
// 16384 cut to 4096: 22.8 us, of which the selection is 11 (20000 cycles, half of them
// the histograms' shared-memory atomics); 513 to 256: 6.8 us.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "ee_cache_ops.cuh"

namespace cg = cooperative_groups;

namespace ee {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 12;
constexpr int kPieces = 4;  // 16-byte pieces of K, and of V, in a thread's registers

// Unsigned integers in the order of the floats, -0 as 0 and NaN below all.
EE_DEV uint32_t order_key(float f) {
  if (isnan(f)) return 0u;
  const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kCopies = 8;

// Shared memory: keys, histograms, kept tokens (16 bits: below 2^14), block tables.
struct Layout {
  int hist, kept, src, dst, bytes;
};
__host__ __device__ inline Layout layout(int max_ctx, int keep) {
  Layout l;
  l.hist = (max_ctx + 3) / 4 * 16;
  l.kept = l.hist + 256 * kCopies * 4;
  l.src = l.kept + (max_ctx * 2 + 15) / 16 * 16;
  l.dst = l.src + (max_ctx + 15) / 16 * 4;
  l.bytes = l.dst + (keep + 15) / 16 * 4;
  return l;
}

template <int HD>
__global__ void __launch_bounds__(kThreads) k_evict(const EvictParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int sums[2][kWarps], s_digit, s_above, s_count;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hkv = p.c.n_kv_heads;
  const int unit = blockIdx.x / C, g = unit % hkv, s = unit / hkv;
  const Layout lay = layout(p.c.max_ctx, p.keep);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
  int* hist = reinterpret_cast<int*>(smem + lay.hist);
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
    constexpr int kFly = 4;  // quarter blocks in flight per thread
    for (int i0 = tid; i0 < (m + 3) / 4; i0 += kFly * kThreads) {
      float4 w[kFly];
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        const int i = min(i0 + u * kThreads, (m + 3) / 4 - 1);
        w[u] = *reinterpret_cast<const float4*>(p.c.weights + ((size_t)max(src[i >> 2], 0) * hkv + g) * 16 + (i & 3) * 4);
      }
#pragma unroll
      for (int u = 0; u < kFly; ++u)
        if (i0 + u * kThreads < (m + 3) / 4)
          reinterpret_cast<uint4*>(keys)[i0 + u * kThreads] =
              make_uint4(order_key(w[u].x), order_key(w[u].y), order_key(w[u].z), order_key(w[u].w));
    }
    uint32_t prefix = 0, mask = 0;
    int rest = need;  // rank of the key looked for, among those that match the prefix
#pragma unroll 1
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
      for (int i = tid; i < 256 * kCopies; i += kThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int t = tid; t < m; t += kThreads) {
        const uint32_t k = keys[t];
        if ((k & mask) == prefix) atomicAdd(&hist[((k >> shift) & 255) * kCopies + lane % kCopies], 1);
      }
      __syncthreads();
      // thread tid < 256: bin 255 - tid, and the keys in the bins above it
      int c = 0, above = 0;
      if (tid < 256) {
#pragma unroll
        for (int u = 0; u < kCopies; ++u) c += hist[(255 - tid) * kCopies + u];
        above = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, above, o);
          if (lane >= o) above += y;
        }
        if (lane == 31) sums[0][warp] = above;
        above -= c;
      }
      __syncthreads();
      if (tid < 256) {
        for (int w = 0; w < warp; ++w) above += sums[0][w];
        if (above < rest && above + c >= rest) {
          s_digit = 255 - tid;
          s_above = above;
          s_count = c;
        }
      }
      __syncthreads();
      rest -= s_above;
      prefix |= (uint32_t)s_digit << shift;
      mask |= 255u << shift;
      if (s_count == rest) break;  // the same for all: every key with this prefix stays
    }
    __syncthreads();
    // Masked keys above prefix stay, the first `rest` equal ones, and the recent
    // tokens.  Warp w owns tokens [t0, t1).
    const int each = (n + kThreads - 1) / kThreads * 32;
    const int t0 = min(n, warp * each), t1 = min(n, t0 + each);
    static_assert(kCacheMaxCtx <= 32 * kThreads, "a warp's run is 32 words of 32 tokens");
    unsigned more = 0, equal = 0;  // of lane i: word i of the run, a bit per token
#pragma unroll 8
    for (int i = 0; i < each / 32; ++i) {
      const uint32_t k = keys[t0 + i * 32 + lane] & mask;  // past the run: other words of shared memory, whose bits go below
      const unsigned a = __ballot_sync(0xffffffffu, k > prefix), e = __ballot_sync(0xffffffffu, k == prefix);
      if (lane == i) {
        more = a;
        equal = e;
      }
    }
    const int word0 = t0 + lane * 32;
    auto before = [&](int t) { return t <= word0 ? 0u : t >= word0 + 32 ? ~0u : (1u << (t - word0)) - 1u; };
    const unsigned cand = need > 0 ? before(min(m, t1)) : 0u;
    equal &= cand;
    more = (more & cand) | (before(t1) & ~before(m));
    int slot = __popc(more), seen = __popc(equal);  // up to and with the word
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, slot, o), y = __shfl_up_sync(0xffffffffu, seen, o);
      if (lane >= o) {
        slot += x;
        seen += y;
      }
    }
    if (lane == 31) {
      sums[0][warp] = slot;
      sums[1][warp] = seen;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
      slot += sums[0][w];
      seen += sums[1][w];
    }
    slot -= __popc(more);  // before the word
    seen -= __popc(equal);
    slot += min(seen, rest);
    for (int over = __popc(equal) - max(0, rest - seen); over > 0; --over) equal &= ~(0x80000000u >> __clz(equal));
    const unsigned stay = more | equal;
#pragma unroll 4
    for (int i = 0; i < each / 32; ++i) {
      const unsigned word = __shfl_sync(0xffffffffu, stay, i);
      const int at = __shfl_sync(0xffffffffu, slot, i) + __popc(word & ((1u << lane) - 1u));
      if (word >> lane & 1) kept[at] = (uint16_t)(t0 + i * 32 + lane);
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
  // Two CTAs per SM, as long as each has a chunk of rows to move.  16384 to 4096 with 8
  // kv heads of 128: 78 us with one CTA per head, 33 with 4, 25 with 8, 23 with 12,
  // and more with 16, too large for some GPCs; 32 sequences of up to 2304 to 1024:
  // 50 us with one, 48 with two, 50 with four.
  const int units = p.batch * p.c.n_kv_heads, chunk = kThreads * kPieces / (HD / 8);
  const int keep = std::min(p.keep, p.c.max_ctx);
  const int C = std::max(1, std::min({kMaxCluster, (2 * sms + units - 1) / units, (keep + chunk - 1) / chunk}));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = layout(p.c.max_ctx, keep).bytes;
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
