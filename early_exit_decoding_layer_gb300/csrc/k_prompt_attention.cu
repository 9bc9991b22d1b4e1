// Causal attention of packed prompt rows over the paged cache: a warp per
// (row, query head) walks the keys once with a running maximum and sum.
#include <math.h>

#include "ee_cache_ops.cuh"

namespace ee {
namespace {

constexpr int kWarps = 8;

template <int HD>
__global__ void __launch_bounds__(kWarps * 32) k_prompt_attention(const PromptParams p) {
  constexpr int E = HD / 32;
  const int s = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
  const int g = h / (p.n_heads / p.c.n_kv_heads);
  const PromptSeq sq = prompt_seq(p, s);
  for (int i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < sq.n; i += gridDim.x * kWarps) {
    const int64_t row = sq.first + i;
    const int last = sq.ctx - sq.n + i;
    float q[E], acc[E], m = -INFINITY, l = 0.0f;
    for (int e = 0; e < E; ++e) {
      q[e] = __half2float(__ushort_as_half(p.q[row * p.q_stride + h * HD + lane * E + e])) * rsqrtf((float)HD);
      acc[e] = 0.0f;
    }
    for (int t = 0; t <= last; ++t) {
      bool ok;
      const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, t, p.c.err, &ok);
      const size_t off = (((size_t)b * p.c.n_kv_heads + g) * 16 + (t & 15)) * HD + lane * E;
      float z = 0.0f;
      for (int e = 0; e < E; ++e) z = fmaf(q[e], __half2float(__ushort_as_half(p.c.k[off + e])), z);
      z = warp_sum(z);
      const float mn = fmaxf(m, z), a = expf(m - mn), w = expf(z - mn);
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * __half2float(__ushort_as_half(p.c.v[off + e]));
      l = l * a + w;
      m = mn;
    }
    const float il = l > 0.0f ? 1.0f / l : 0.0f;
    for (int e = 0; e < E; ++e) p.o[row * p.o_stride + h * HD + lane * E + e] = float_to_half_bits(acc[e] * il);
    if (p.lse && lane == 0) p.lse[(size_t)h * p.total_q + row] = m + logf(l);
  }
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptParams& p, cudaStream_t st) {
  const dim3 grid((p.total_q + kWarps - 1) / kWarps, p.n_heads, p.n_seqs);
  if (p.c.head_dim == 64)
    k_prompt_attention<64><<<grid, kWarps * 32, 0, st>>>(p);
  else
    k_prompt_attention<128><<<grid, kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace ee
