// What each cached token weighs in the attention of packed prompt rows: a warp
// per (token, kv head) walks the rows that see it.
#include <math.h>

#include "ee_cache_ops.cuh"

namespace ee {
namespace {

constexpr int kWarps = 8;

template <int HD>
__global__ void __launch_bounds__(kWarps * 32) k_prompt_weights(const PromptParams p) {
  constexpr int E = HD / 32;
  const int s = blockIdx.z, g = blockIdx.y, lane = threadIdx.x & 31, G = p.n_heads / p.c.n_kv_heads;
  const PromptSeq sq = prompt_seq(p, s);
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= sq.ctx) return;
  bool ok;
  const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, t, p.c.err, &ok);
  const size_t slot = ((size_t)b * p.c.n_kv_heads + g) * 16 + (t & 15);
  float k[E], w = 0.0f;
  for (int e = 0; e < E; ++e) k[e] = __half2float(__ushort_as_half(p.c.k[slot * HD + lane * E + e])) * rsqrtf((float)HD);
  for (int i = max(0, t - (sq.ctx - sq.n)); i < sq.n; ++i)
    for (int h = g * G; h < (g + 1) * G; ++h) {
      const int64_t row = sq.first + i;
      float z = 0.0f;
      for (int e = 0; e < E; ++e)
        z = fmaf(k[e], __half2float(__ushort_as_half(p.q[row * p.q_stride + h * HD + lane * E + e])), z);
      z = warp_sum(z);
      const float lse = p.lse_in[(size_t)h * p.total_q + row];
      if (lse != -INFINITY) w += expf(z - lse);
    }
  if (lane == 0 && ok) atomicAdd(p.c.weights + slot, w);
}

}  // namespace

cudaError_t launch_prompt_weights(const PromptParams& p, cudaStream_t st) {
  const dim3 grid((p.c.max_ctx + kWarps - 1) / kWarps, p.c.n_kv_heads, p.n_seqs);
  if (p.c.head_dim == 64)
    k_prompt_weights<64><<<grid, kWarps * 32, 0, st>>>(p);
  else
    k_prompt_weights<128><<<grid, kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace ee
