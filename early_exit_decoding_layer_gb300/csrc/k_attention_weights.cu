// Decode attention over the paged cache that adds each token's weight: a CTA
// per (sequence, kv head), scores kept in shared memory.
#include <math.h>

#include "ee_cache_ops.cuh"

namespace ee {
namespace {

constexpr int kWarps = 8;

// Query heads one after another, so that one row of scores fits.
template <int HD>
__global__ void __launch_bounds__(kWarps * 32) k_attention_weights(const DecodeWeightsParams p) {
  constexpr int E = HD / 32;
  extern __shared__ float sc[];  // [max_ctx]
  __shared__ float red[kWarps], part[kWarps][HD];
  const int g = blockIdx.x, s = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.n_heads / p.c.n_kv_heads;
  const int n = checked_length(p.pos[s] == INT32_MAX ? INT32_MAX : p.pos[s] + 1, p.c.max_ctx, p.c.err);
  bool ok;
  for (int h = g * G; h < (g + 1) * G; ++h) {
    float q[E], acc[E], m = -INFINITY;
    const float* qp = p.q + ((size_t)s * p.n_heads + h) * HD + lane * E;
    for (int e = 0; e < E; ++e) q[e] = qp[e] * rsqrtf((float)HD), acc[e] = 0.0f;
    for (int t = warp; t < n; t += kWarps) {
      const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, t, p.c.err, &ok);
      const size_t slot = ((size_t)b * p.c.n_kv_heads + g) * 16 + (t & 15);
      float z = 0.0f;
      for (int e = 0; e < E; ++e) z = fmaf(q[e], __half2float(__ushort_as_half(p.c.k[slot * HD + lane * E + e])), z);
      z = warp_sum(z);
      m = fmaxf(m, z);
      if (lane == 0) sc[t] = z;
    }
    if (lane == 0) red[warp] = m;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, red[w]);
    __syncthreads();
    float l = 0.0f;
    for (int t = warp; t < n; t += kWarps) {
      const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, t, p.c.err, &ok);
      const size_t slot = ((size_t)b * p.c.n_kv_heads + g) * 16 + (t & 15);
      const float e0 = expf(sc[t] - m);
      l += e0;
      for (int e = 0; e < E; ++e)
        acc[e] = fmaf(e0, __half2float(__ushort_as_half(p.c.v[slot * HD + lane * E + e])), acc[e]);
    }
    for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
    if (lane == 0) red[warp] = l;
    __syncthreads();
    l = 0.0f;
    for (int w = 0; w < kWarps; ++w) l += red[w];
    const float il = n > 0 ? 1.0f / l : 0.0f;
    for (int i = threadIdx.x; i < HD; i += blockDim.x) {
      float a = 0.0f;
      for (int w = 0; w < kWarps; ++w) a += part[w][i];
      p.o[((size_t)s * p.n_heads + h) * HD + i] = a * il;
    }
    for (int t = threadIdx.x; t < n; t += blockDim.x) {
      const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, t, p.c.err, &ok);
      if (ok) atomicAdd(p.c.weights + ((size_t)b * p.c.n_kv_heads + g) * 16 + (t & 15), expf(sc[t] - m) * il);
    }
    __syncthreads();
  }
}

template <int HD>
cudaError_t launch_t(const DecodeWeightsParams& p, cudaStream_t st) {
  const size_t smem = (size_t)p.c.max_ctx * 4;
  const cudaError_t e =
      cudaFuncSetAttribute(k_attention_weights<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheMaxCtx * 4);
  if (e != cudaSuccess) return e;
  k_attention_weights<HD><<<dim3(p.c.n_kv_heads, p.batch), kWarps * 32, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_weights(const DecodeWeightsParams& p, cudaStream_t st) {
  return p.c.head_dim == 64 ? launch_t<64>(p, st) : launch_t<128>(p, st);
}

}  // namespace ee
