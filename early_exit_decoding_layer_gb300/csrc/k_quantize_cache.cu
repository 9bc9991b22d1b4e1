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
// half a row stand side by side.  Memory is the bound: 35000 tokens of 8 heads of 128 written in
// 36.5 us (5.9 TB/s), from fp32 rows in 55.9 (6.4 TB/s), 37000 read back in 38.6 us (5.9 TB/s); one
// token 2.2 us, the launch.
#include "ee_cache_ops.cuh"
#include "ee_tcgen05.cuh"

namespace ee {
namespace {

constexpr int kThreads = 128;
constexpr int kMinExponent = -15;
constexpr float kHalfEnd = 65520.0f;  // from here on fp16 rounds to infinity

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

// A warp has a row: where it goes is found once for all of its heads, of which 256 / HD stand
// side by side, HD / 8 lanes each, U of these steps in flight.  (With a search, a
// division and a table entry for every head instructions were the bound: 36000 rows of 8 heads of
// 128 in fp16 took 49 us, then 39.)  U = 4 in fp16 has few warps per SM: it is for calls whose
// rows are all on their way at once (8 heads of 128, 64 rows: 2.7 us, with U = 2 3.0; 2048: 4.0, 4.2);
// others are faster with U = 2 and registers for ten CTAs per SM (8192 rows: 11.0 us, with U = 4
// 11.9; 35000: 36.5, 39).  fp32 rows are twice the bytes in flight with U = 2 (64: 3.3 us, 2048: 5.2,
// 8192: 15.2).
template <typename T, int HD, int U>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && U == 2 ? 10 : 1) k_quantize_cache(const QuantizeParams p) {
  constexpr int L = HD / 8, kHeads = 32 / L;
  const int lane = threadIdx.x & 31, col = (lane % L) * 8, hkv = p.c.n_kv_heads;
  const int row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= p.total) return;
  const T *k = static_cast<const T*>(p.k) + row * p.k_stride + col, *v = static_cast<const T*>(p.v) + row * p.v_stride + col;
  Eight<T> x[U][2];
  auto load = [&](int g0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * kHeads + lane / L;
      if (g < hkv) {
        x[u][0].load(k + g * HD);
        x[u][1].load(v + g * HD);
      } else {
        x[u][0].clear();
        x[u][1].clear();
      }
    }
  };
  load(0);
  // the row's sequence is the first that ends behind it
  static_assert(EE_MAX_BATCH <= 64, "two sequences per lane");
  const int n = p.n_seqs, end0 = lane < n ? p.cu[lane + 1] : INT32_MAX, end1 = lane + 32 < n ? p.cu[lane + 33] : INT32_MAX;
  const int first = p.cu[0];
  const unsigned b0 = __ballot_sync(0xffffffffu, end0 > row), b1 = __ballot_sync(0xffffffffu, end1 > row);
  const int s = b0 ? __ffs(b0) - 1 : b1 ? 31 + __ffs(b1) : 64;
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    int prev0 = __shfl_up_sync(0xffffffffu, end0, 1), prev1 = __shfl_up_sync(0xffffffffu, end1, 1);
    const int last0 = __shfl_sync(0xffffffffu, end0, 31);
    if (lane == 0) {
      prev0 = first;
      prev1 = last0;
    }
    if ((lane < n && (end0 < prev0 || end0 < 0 || end0 > p.total)) || (lane + 32 < n && (end1 < prev1 || end1 < 0 || end1 > p.total)) ||
        first < 0 || first > p.total)
      report(p.c.err, EE_DERR_LENGTH);
  }
  int64_t to = -1;  // (block, slot)
  int slot = 0;
  if (s < n && p.cu[s] <= row) {
    const int64_t pos = (int64_t)checked_length(p.ctx[s], p.c.max_ctx, p.c.err) - p.cu[s + 1] + row;
    if (pos >= 0) {
      bool ok;
      const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, s, (int)pos, p.c.err, &ok);
      if (ok) to = b;
      slot = (int)pos & 15;
    }
  }
  if (to < 0) return;
  for (int g0 = 0; g0 < hkv; g0 += U * kHeads) {
    if (g0 > 0) load(g0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * kHeads + lane / L;
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
        if (g < hkv) {
          const int64_t at = ((to * hkv + g) * 2 + kv) * 16 + slot;
          *reinterpret_cast<uint2*>(p.codes + at * HD + col) = w;
          if (col == 0) p.exponents[at] = (int8_t)e;
        }
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
  const int n = (p.total + kThreads / 32 - 1) / (kThreads / 32);
  // U = 4 is of no use where the heads of a row fit into a step of two
  bool four = false;
  if (sizeof(T) == 2 && p.c.n_kv_heads > 2 * (256 / HD)) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    four = p.total <= 24 * sms;  // rows at once, 24 warps per SM
  }
  if (four) k_quantize_cache<T, HD, sizeof(T) == 2 ? 4 : 2><<<n, kThreads, 0, st>>>(p);
  else k_quantize_cache<T, HD, 2><<<n, kThreads, 0, st>>>(p);
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
