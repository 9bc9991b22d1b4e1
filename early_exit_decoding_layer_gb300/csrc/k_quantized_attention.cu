// Decode attention over the eight-bit cache: a warp per sequence and query head walks
// the tokens with a running maximum and sum, hd / 32 dims a lane.
#include <math.h>

#include "ee_cache_ops.cuh"
#include "ee_tcgen05.cuh"

namespace ee {
namespace {

EE_DEV float from_e4m3(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

template <int HD>
__global__ void k_quantized_attention(const DecodeParams p) {
  constexpr int N = HD / 32;
  const int lane = threadIdx.x & 31, at = blockIdx.x * 4 + (threadIdx.x >> 5), hkv = p.c.n_kv_heads;
  if (at >= p.batch * p.n_heads) return;
  const int s = at / p.n_heads, h = at % p.n_heads, g = h / (p.n_heads / hkv);
  const int ctx = checked_length(p.pos[s] == INT32_MAX ? INT32_MAX : p.pos[s] + 1, p.c.max_ctx, p.c.err);
  float q[N], o[N], m = -INFINITY, l = 0.0f;
  for (int i = 0; i < N; ++i) {
    q[i] = __half2float(__ushort_as_half(p.q[s * p.q_stride + h * HD + i * 32 + lane])) * (1.4426950408889634f / sqrtf((float)HD));
    if (isinf(q[i])) q[i] = NAN;
    o[i] = 0.0f;
  }
  for (int t = 0; t < ctx; ++t) {
    bool ok;
    const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, t, p.c.err, &ok);
    const int64_t k = ((int64_t)b * hkv + g) * 32 + (t & 15), v = k + 16;
    float z = 0.0f;
    for (int i = 0; i < N; ++i) z += q[i] * from_e4m3(p.codes[k * HD + i * 32 + lane]);
    z = warp_sum(z) * exp2f((float)p.exponents[k]);
    const float mn = fmaxf(m, z), a = ex2(m - mn), e = ex2(z - mn), w = e * exp2f((float)p.exponents[v]);
    m = mn;
    l = l * a + e;
    for (int i = 0; i < N; ++i) o[i] = o[i] * a + w * from_e4m3(p.codes[v * HD + i * 32 + lane]);
  }
  for (int i = 0; i < N; ++i) {
    const float x = ctx > 0 ? o[i] / l : 0.0f;
    p.o[s * p.o_stride + h * HD + i * 32 + lane] =
        float_to_half_bits(fabsf(x) < INFINITY ? fminf(fmaxf(x, -65504.0f), 65504.0f) : x);
  }
}

}  // namespace

cudaError_t launch_quantized_attention(const DecodeParams& p, cudaStream_t st) {
  const unsigned n = (unsigned)(p.batch * p.n_heads + 3) / 4;
  if (p.c.head_dim == 64) k_quantized_attention<64><<<n, 128, 0, st>>>(p);
  else k_quantized_attention<128><<<n, 128, 0, st>>>(p);
  return cudaGetLastError();
}

size_t quantized_attention_scratch(int32_t, int32_t, int32_t, int32_t, int32_t) { return 16; }

}  // namespace ee
