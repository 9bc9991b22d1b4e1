// The eight-bit cache's writing and reading back.
//
// A row of K or V (one token, one kv head) is held as e4m3 codes times 2^e, e the least
// exponent with which its largest value is within e4m3's 448.  In a floating format a
// scale that fits more closely gains nothing: a code has four significant bits at
// any scale, so a power of two costs at most one binade of the 15 below the largest
// value, multiplies exactly, and reads back as an fp16 value.  e is -15 or more, which is
// where a code's last bit becomes fp16's own, 2^-24.
//
// Both kernels stream: eight values a thread, so that 16-byte (or two) loads and stores of
// half a row stand side by side.
#include "ee_cache_ops.cuh"
#include "ee_tcgen05.cuh"

namespace ee {
namespace {

constexpr int kThreads = 256;
constexpr int kMinExponent = -15;
constexpr float kHalfEnd = 65520.0f;  // from here on fp16 rounds to infinity

// Two values as e4m3, the first in the low byte.
EE_DEV uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}

EE_DEV float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Eight values of a row in registers, 16 or 32 bytes.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  uint4 a;
  EE_DEV void load(const uint16_t* p) { a = ldg_stream_v4(p); }
  EE_DEV void clear() { a = make_uint4(0, 0, 0, 0); }
  EE_DEV void values(float* x) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Eight<float> {
  uint4 a, b;
  EE_DEV void load(const float* p) {
    a = ldg_stream_v4(p);
    b = ldg_stream_v4(p + 4);
  }
  EE_DEV void clear() { a = b = make_uint4(0, 0, 0, 0); }
  EE_DEV void values(float* x) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
};

// HD / 8 threads to a (row, kv head), K and V; kItems of these a step.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) k_quantize_cache(const QuantizeParams p) {
  constexpr int L = HD / 8, kItems = kThreads / L, U = 2;
  __shared__ int cu[EE_MAX_BATCH + 1];
  const int tid = threadIdx.x, col = (tid % L) * 8, hkv = p.c.n_kv_heads;
  const int64_t items = (int64_t)p.total * hkv, first = (int64_t)blockIdx.x * kItems * U + tid / L;
  Eight<T> x[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t item = first + u * kItems;
    const int64_t row = item / hkv, at = (item - row * hkv) * HD + col;
    if (item < items) {
      x[u][0].load(static_cast<const T*>(p.k) + row * p.k_stride + at);
      x[u][1].load(static_cast<const T*>(p.v) + row * p.v_stride + at);
    } else {
      x[u][0].clear();
      x[u][1].clear();
    }
  }
  if (tid <= p.n_seqs) cu[tid] = p.cu[tid];
  __syncthreads();
  if (blockIdx.x == 0 && tid <= p.n_seqs && (cu[tid] < 0 || cu[tid] > p.total || (tid > 0 && cu[tid] < cu[tid - 1])))
    report(p.c.err, EE_DERR_LENGTH);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t item = first + u * kItems;
    const int row = (int)(item / hkv), g = (int)(item - (int64_t)row * hkv);
    // the first sequence that ends behind the row
    int s = 0, end = p.n_seqs;
    while (s < end) {
      const int mid = (s + end) >> 1;
      if (cu[mid + 1] > row) end = mid;
      else s = mid + 1;
    }
    int64_t to = -1;  // (block, head)
    int slot = 0;
    if (item < items && s < p.n_seqs && cu[s] <= row) {
      const int64_t pos = (int64_t)checked_length(p.ctx[s], p.c.max_ctx, p.c.err) - cu[s + 1] + row;
      if (pos >= 0) {
        bool ok;
        const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, (int)pos, p.c.err, &ok);
        if (ok) to = (int64_t)b * hkv + g;
        slot = (int)pos & 15;
      }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float y[8], big = 0.0f;
      x[u][kv].values(y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!(fabsf(y[i]) < kHalfEnd)) y[i] = __uint_as_float(0x7fffffffu);
        big = fmaxf(big, fabsf(y[i]));  // of a number and NaN the number
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      // big = 1.f * 2^E; 448 = 1.75 * 2^8
      const uint32_t bits = __float_as_uint(big);
      const int e = max(kMinExponent, (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0));
      const float down = pow2(-e);
      uint2 w;
      w.x = to_e4m3x2(y[0] * down, y[1] * down) | to_e4m3x2(y[2] * down, y[3] * down) << 16;
      w.y = to_e4m3x2(y[4] * down, y[5] * down) | to_e4m3x2(y[6] * down, y[7] * down) << 16;
      if (to >= 0) {
        const int64_t at = (to * 2 + kv) * 16 + slot;
        *reinterpret_cast<uint2*>(p.codes + at * HD + col) = w;
        if (col == 0) p.exponents[at] = (int8_t)e;
      }
    }
  }
}

// A CTA reads up to kThreads * U pieces of eight codes of one block: all of it where it
// has few heads, else some of its heads (blockIdx.z).
template <int HD>
__global__ void __launch_bounds__(kThreads) k_dequantize_cache(const DequantizeParams p) {
  constexpr int L = HD / 8, U = 4;  // pieces per row; pieces per thread
  const int s = blockIdx.y, b = blockIdx.x, tid = threadIdx.x, hkv = p.c.n_kv_heads;
  const int live = checked_length(p.ctx[s], p.c.max_ctx, p.c.err) - b * 16;  // slots that hold a token
  if (live <= 0) return;
  bool ok, to_ok;
  const int src = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, b * 16, p.c.err, &ok);
  const int dst = checked_block(p.dst_table, p.dst_stride, p.n_dst, s, b * 16, p.c.err, &to_ok);
  if (!ok || !to_ok) return;
  const int pieces = hkv * 32 * L, first = blockIdx.z * kThreads * U + tid;
  uint2 w[U];
  int e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = first + u * kThreads, row = i / L;  // row: head, K or V, slot
    if (i < pieces && (row & 15) < live) {
      const int64_t at = (int64_t)src * hkv * 32 + row;
      w[u] = *reinterpret_cast<const uint2*>(p.codes + at * HD + (i % L) * 8);
      e[u] = p.exponents[at];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = first + u * kThreads, row = i / L;
    if (i < pieces && (row & 15) < live) {
      // code * 2^e is exact in fp16 but for 65536 (and infinities are of overflow alone)
      const __half up = __ushort_as_half((unsigned short)(e[u] >= -14 ? (15 + e[u]) << 10 : 1 << 9));
      const __half2 up2 = __halves2half2(up, up), most = __float2half2_rn(65504.0f), least = __float2half2_rn(-65504.0f);
      const uint32_t c[4] = {w[u].x & 0xffffu, w[u].x >> 16, w[u].y & 0xffffu, w[u].y >> 16};
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c[k]));
        __half2 y = __hmul2(*reinterpret_cast<__half2*>(&h), up2);
        y = __hmax2_nan(__hmin2_nan(y, most), least);
        r[k] = *reinterpret_cast<uint32_t*>(&y);
      }
      uint16_t* to = (row & 16) ? p.v : p.k;
      const int64_t at = ((int64_t)dst * hkv + (row >> 5)) * 16 + (row & 15);
      *reinterpret_cast<uint4*>(to + at * HD + (i % L) * 8) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
}

template <typename T, int HD>
cudaError_t quantize_t(const QuantizeParams& p, cudaStream_t st) {
  const int64_t each = kThreads / (HD / 8) * 2, n = ((int64_t)p.total * p.c.n_kv_heads + each - 1) / each;
  if (n > INT32_MAX) return cudaErrorInvalidValue;
  k_quantize_cache<T, HD><<<(unsigned)n, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int HD>
cudaError_t dequantize_t(const DequantizeParams& p, cudaStream_t st) {
  const int pieces = p.c.n_kv_heads * 32 * (HD / 8), each = kThreads * 4;
  const dim3 grid((p.c.max_ctx + 15) / 16, p.batch, (pieces + each - 1) / each);
  k_dequantize_cache<HD><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_cache(const QuantizeParams& p, cudaStream_t st) {
  if (p.c.head_dim == 64) return p.rows_type == EE_ROWS_F32 ? quantize_t<float, 64>(p, st) : quantize_t<uint16_t, 64>(p, st);
  return p.rows_type == EE_ROWS_F32 ? quantize_t<float, 128>(p, st) : quantize_t<uint16_t, 128>(p, st);
}

cudaError_t launch_dequantize_cache(const DequantizeParams& p, cudaStream_t st) {
  return p.c.head_dim == 64 ? dequantize_t<64>(p, st) : dequantize_t<128>(p, st);
}

}  // namespace ee
