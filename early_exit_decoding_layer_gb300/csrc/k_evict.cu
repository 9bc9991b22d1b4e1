// Eviction from the paged cache by accumulated weight.
//
// Per (sequence, kv head): the keep - recent heaviest of the tokens before the
// last `recent` are found by a radix selection over the weights' bits, mapped to
// unsigned integers of the same order (four passes of 8 bits: a histogram,
// its suffix sums, the digit in which the wanted rank falls).  Tokens
// above the resulting key stay, and of those equal to it the first ones, so ties
// go to the lower index.  A prefix sum over the flags gives every kept token
// its slot.  Slots are never above their tokens, so the rows can move in place
// in ascending order: a chunk of rows is read into registers, all threads
// meet, and it is written; later chunks read only rows behind it.
#include <math.h>

#include "ee_cache_ops.cuh"

namespace ee {
namespace {

constexpr int kThreads = 512;

// Unsigned integers in the order of the floats, -0 as 0 and NaN below all.
EE_DEV uint32_t order_key(float f) {
  if (isnan(f)) return 0u;
  const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of one value per thread, and the total.
EE_DEV int block_scan(int v, int* warps, int* total) {
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
  int base = 0, sum = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += warps[w];
    sum += warps[w];
  }
  *total = sum;
  return base + x - v;
}

template <int HD>
__global__ void __launch_bounds__(kThreads) k_evict(const EvictParams p) {
  extern __shared__ uint32_t keys[];  // [max_ctx], then the kept tokens [max_ctx]
  int32_t* kept = reinterpret_cast<int32_t*>(keys + p.c.max_ctx);
  __shared__ int hist[256], warps[kThreads / 32], s_digit, s_above;
  const int g = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, hkv = p.c.n_kv_heads;
  const int n = checked_length(p.ctx[s], p.c.max_ctx, p.c.err);
  const int len = min(n, p.keep);
  if (g == 0 && tid == 0) p.new_ctx[s] = len;
  bool ok;
  if (n <= p.keep) {
    for (int i = tid; i < n; i += kThreads) kept[i] = i;
  } else {
    const int m = n - p.recent;     // candidates
    const int need = p.keep - p.recent;  // < m
    for (int t = tid; t < m; t += kThreads) {
      const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, t, p.c.err, &ok);
      keys[t] = order_key(p.c.weights[((size_t)b * hkv + g) * 16 + (t & 15)]);
    }
    uint32_t prefix = 0, mask = 0;
    int rank = need;  // the rank-th largest among the keys that match the prefix
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int t = tid; t < m; t += kThreads)
        if ((keys[t] & mask) == prefix) atomicAdd(&hist[(keys[t] >> shift) & 255], 1);
      __syncthreads();
      if (tid == 0) {
        int above = 0, d = 255;
        while (above + hist[d] < rank) above += hist[d--];
        s_digit = d;
        s_above = above;
      }
      __syncthreads();
      rank -= s_above;
      prefix |= (uint32_t)s_digit << shift;
      mask |= 255u << shift;
      __syncthreads();
    }
    // keys above `prefix` stay, and the first `rank` that equal it
    int base = 0, ties = 0;
    for (int t0 = 0; t0 < n; t0 += kThreads) {
      const int t = t0 + tid;
      const bool cand = t < m, eq = cand && need > 0 && keys[t] == prefix;
      int total;
      const int e = block_scan(eq, warps, &total) + ties;
      ties += total;
      const bool stay = (t >= m && t < n) || (cand && need > 0 && (keys[t] > prefix || (eq && e < rank)));
      const int at = block_scan(stay, warps, &total) + base;
      base += total;
      if (stay) kept[at] = t;
    }
  }
  __syncthreads();
  if (p.kept)
    for (int i = tid; i < p.keep; i += kThreads) p.kept[((size_t)s * hkv + g) * p.keep + i] = i < len ? kept[i] : -1;
  if (n <= p.keep && p.dst_table == p.c.table) return;  // in place already
  // rows move in ascending order, a thread per 16-byte piece of K and V
  constexpr int PIECES = HD / 8;
  const uint4* kc = reinterpret_cast<const uint4*>(p.c.k);
  const uint4* vc = reinterpret_cast<const uint4*>(p.c.v);
  for (int i0 = 0; i0 < len; i0 += kThreads / PIECES) {
    const int i = i0 + tid / PIECES, j = tid % PIECES;
    uint4 a, b;
    float w;
    bool dst_ok = false;
    size_t dst = 0;
    if (i < len) {
      const int t = kept[i];
      const int sb = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, t, p.c.err, &ok);
      const int db = checked_block(p.dst_table, p.dst_stride, p.c.n_blocks, s, i, p.c.err, &dst_ok);
      const size_t src = ((size_t)sb * hkv + g) * 16 + (t & 15);
      dst = ((size_t)db * hkv + g) * 16 + (i & 15);
      a = kc[src * PIECES + j];
      b = vc[src * PIECES + j];
      w = p.c.weights[src];
    }
    __syncthreads();
    if (dst_ok) {
      const_cast<uint4*>(kc)[dst * PIECES + j] = a;
      const_cast<uint4*>(vc)[dst * PIECES + j] = b;
      if (j == 0) p.c.weights[dst] = w;
    }
  }
}

template <int HD>
cudaError_t launch_t(const EvictParams& p, cudaStream_t st) {
  const size_t smem = (size_t)p.c.max_ctx * 8;
  const cudaError_t e =
      cudaFuncSetAttribute(k_evict<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheMaxCtx * 8);
  if (e != cudaSuccess) return e;
  k_evict<HD><<<dim3(p.c.n_kv_heads, p.batch), kThreads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t st) {
  return p.c.head_dim == 64 ? launch_t<64>(p, st) : launch_t<128>(p, st);
}

}  // namespace ee
