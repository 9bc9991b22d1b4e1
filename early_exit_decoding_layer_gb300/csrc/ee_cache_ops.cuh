// Parameters and launchers of the operators on the paged cache: attention of
// packed prompt rows, the weights of its tokens, decode attention that adds
// weights, eviction; the eight-bit cache's writing, reading back and decode
// attention; decode attention behind a shared prefix.  Lengths and block ids come from device memory and are
// checked here, in the kernels: what is out of range is cut to the range and
// reported in the error word.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ee.h"
#include "ee_common.cuh"

namespace ee {

constexpr int kCacheMaxCtx = 16384;

// One layer's cache and the sequences' block tables.
struct PagedCache {
  const uint16_t* k = nullptr;
  const uint16_t* v = nullptr;
  float* weights = nullptr;
  const int32_t* table = nullptr;
  int32_t table_stride = 0;
  int32_t n_blocks = 0;
  int32_t n_kv_heads = 0;
  int32_t head_dim = 0;
  int32_t max_ctx = 0;  // at most 16 * table_stride
  int32_t* err = nullptr;
};

// Packed prompt rows (prompt attention and prompt weights).
struct PromptParams {
  PagedCache c;
  int32_t n_seqs = 0, total_q = 0, n_heads = 0;
  const uint16_t* q = nullptr;
  int64_t q_stride = 0;
  const int32_t* cu_q = nullptr;
  const int32_t* ctx = nullptr;
  uint16_t* o = nullptr;
  int64_t o_stride = 0;
  const float* lse_in = nullptr;  // weights
  float* lse = nullptr;           // attention
};

struct DecodeWeightsParams {
  PagedCache c;
  int32_t batch = 0, n_heads = 0;
  const float* q = nullptr;
  const int32_t* pos = nullptr;
  float* o = nullptr;
};

struct EvictParams {
  PagedCache c;
  int32_t batch = 0, keep = 0, recent = 0;
  const int32_t* dst_table = nullptr;  // the source table: in place
  int32_t dst_stride = 0;
  const int32_t* ctx = nullptr;
  int32_t* new_ctx = nullptr;
  int32_t* kept = nullptr;
};

// The eight-bit cache: codes [n_blocks, Hkv, 2, 16, hd], exponents [n_blocks, Hkv, 2, 16].
struct QuantizeParams {
  PagedCache c;  // k, v, weights unused
  uint8_t* codes = nullptr;
  int8_t* exponents = nullptr;
  int32_t n_seqs = 0, total = 0, rows_type = 0;
  const void* k = nullptr;
  const void* v = nullptr;
  int64_t k_stride = 0, v_stride = 0;  // in elements
  const int32_t* cu = nullptr;
  const int32_t* ctx = nullptr;
};

struct DequantizeParams {
  PagedCache c;  // k, v, weights unused
  const uint8_t* codes = nullptr;
  const int8_t* exponents = nullptr;
  int32_t batch = 0;
  const int32_t* ctx = nullptr;
  uint16_t* k = nullptr;
  uint16_t* v = nullptr;
  int32_t n_dst = 0;
  const int32_t* dst_table = nullptr;
  int32_t dst_stride = 0;
};

// One query row per sequence, fp16 in and out.
struct DecodeParams {
  PagedCache c;
  const uint8_t* codes = nullptr;  // of the eight-bit cache; else c.k and c.v
  const int8_t* exponents = nullptr;
  int32_t batch = 0, n_heads = 0, prefix = 0;  // prefix in whole blocks' tokens, at most c.max_ctx of them
  const uint16_t* q = nullptr;
  int64_t q_stride = 0;
  const int32_t* pos = nullptr;
  uint16_t* o = nullptr;
  int64_t o_stride = 0;
  void* scratch = nullptr;
};

// exp(z - x) of a score z = q . k / sqrt(hd), from the tensor core's sum s, as
// 2^(c s - f x): c is log2(e) / sqrt(hd) rounded to fp32 and f c's counterpart in two
// terms, so that c's rounding multiplies z - x and not z and x each (1e-6 at a
// score of 10 otherwise).  unit is 1 / sqrt(hd) in two terms.
//
// The tensor core's accumulator is cut, not rounded, after each of the hd / 16 steps of
// a product, so sums come out smaller by about 0.42 * 2^-23 of each partial
// sum (hd 128: 2.1e-7 of s measured, hd 64: 1.4e-7; weights of tokens with
// z = 6 were 1.2e-6 too small).  c, f and unit take that mean back.
struct Exponent {
  float c, f_hi, f_lo, unit_hi, unit_lo;
};
inline Exponent make_exponent(int head_dim) {
  const double r = sqrt((double)head_dim);
  const double grow = 1.0 + 0.42 * 0x1p-23 * (head_dim / 16 + 1) / 2;  // partial sums grow evenly
  Exponent e;
  e.c = (float)(1.4426950408889634074 * grow / r);
  const double f = (double)e.c * r / grow, unit = grow / r;
  e.f_hi = (float)f;
  e.f_lo = (float)(f - e.f_hi);
  e.unit_hi = (float)unit;
  e.unit_lo = (float)(unit - e.unit_hi);
  return e;
}

cudaError_t launch_prompt_attention(const PromptParams& p, cudaStream_t st);
cudaError_t launch_prompt_weights(const PromptParams& p, cudaStream_t st);
cudaError_t launch_attention_weights(const DecodeWeightsParams& p, cudaStream_t st);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t st);
cudaError_t launch_quantize_cache(const QuantizeParams& p, cudaStream_t st);
cudaError_t launch_dequantize_cache(const DequantizeParams& p, cudaStream_t st);
cudaError_t launch_quantized_attention(const DecodeParams& p, cudaStream_t st);
cudaError_t launch_shared_attention(const DecodeParams& p, cudaStream_t st);
size_t quantized_attention_scratch(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_ctx);
size_t shared_attention_scratch(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_ctx,
                                int32_t prefix);

#ifdef __CUDACC__
// o is a mean of the values that the cache holds and no larger than they are.  Its rounding on the way
// may take it past the largest one, which would be infinite in fp16.
constexpr float kMostHalf = 65504.0f;
EE_DEV float within_half(float y) {
  return fabsf(y) > kMostHalf && fabsf(y) < INFINITY ? copysignf(kMostHalf, y) : y;
}

// Two values as e4m3, the first in the low byte.
EE_DEV uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}

EE_DEV float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

EE_DEV void report(int32_t* err, int32_t code) {
  if (err) atomicCAS(err, 0, code);
}

// A length from device memory, cut to [0, most].
EE_DEV int checked_length(int n, int most, int32_t* err) {
  if (n < 0 || n > most) {
    report(err, EE_DERR_LENGTH);
    n = n < 0 ? 0 : most;
  }
  return n;
}

// The block of token t of sequence s; *ok false and block 0 if its id is out
// of range.
EE_DEV int checked_block(const int32_t* table, int64_t stride, int n_blocks, int s, int t, int32_t* err, bool* ok) {
  int b = table[s * stride + (t >> 4)];
  *ok = b >= 0 && b < n_blocks;
  if (!*ok) {
    report(err, EE_DERR_BLOCK);
    b = 0;
  }
  return b;
}

// Rows [first, first + n) and cached tokens of packed sequence s.
struct PromptSeq {
  int first, n, ctx;
};
EE_DEV PromptSeq prompt_seq(const PromptParams& p, int s) {
  PromptSeq r;
  r.first = checked_length(p.cu_q[s], p.total_q, p.c.err);
  const int end = checked_length(p.cu_q[s + 1], p.total_q, p.c.err);
  if (end < r.first) report(p.c.err, EE_DERR_LENGTH);
  r.n = end > r.first ? end - r.first : 0;
  r.ctx = checked_length(p.ctx[s], p.c.max_ctx, p.c.err);
  return r;
}

// Tiles of `rows` rows of every sequence, numbered so that those with the most keys
// come first (they are started first): a tile's level is its last row's
// position over `rows`, levels count down, and within a level the sequences
// count up.  A whole warp holds the index, two sequences per lane.
struct PromptTile {
  int s, i0;  // sequence (-1: there is no such tile), the tile's first row within it
  PromptSeq sq;
};
struct PromptIndex {
  PromptSeq sq[2];
  int base[2], end[2], top, rows;

  EE_DEV void init(const PromptParams& p, int rows_) {
    static_assert(EE_MAX_BATCH <= 64, "two sequences per lane");
    rows = rows_;
    top = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int s = (threadIdx.x & 31) + 32 * u;
      sq[u] = s < p.n_seqs ? prompt_seq(p, s) : PromptSeq{0, 0, 0};
      base[u] = max(0, sq[u].ctx - sq[u].n) / rows;
      end[u] = base[u] + (sq[u].n + rows - 1) / rows;
      top = max(top, end[u]);
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  // tiles at level l or above
  EE_DEV int above(int l) const {
    const int c = max(end[0] - max(base[0], l), 0) + max(end[1] - max(base[1], l), 0);
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)c);
  }
  EE_DEV PromptTile find(int rank) const {
    PromptTile r = {-1, 0, {0, 0, 0}};
    if (rank >= above(0)) return r;
    int lo = 0, hi = top;  // above(lo) > rank >= above(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (above(mid) > rank) lo = mid;
      else hi = mid;
    }
    int idx = rank - above(hi);  // the idx-th sequence with a tile at level lo
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool has = base[u] <= lo && lo < end[u];
      const unsigned m = __ballot_sync(0xffffffffu, has);
      const int lane = threadIdx.x & 31;
      const unsigned hit = __ballot_sync(0xffffffffu, has && __popc(m & ((1u << lane) - 1u)) == idx);
      if (hit && r.s < 0) {
        const int src = __ffs(hit) - 1;
        r.s = src + 32 * u;
        r.i0 = (lo - __shfl_sync(0xffffffffu, base[u], src)) * rows;
        r.sq.first = __shfl_sync(0xffffffffu, sq[u].first, src);
        r.sq.n = __shfl_sync(0xffffffffu, sq[u].n, src);
        r.sq.ctx = __shfl_sync(0xffffffffu, sq[u].ctx, src);
      }
      idx -= __popc(m);
    }
    return r;
  }
};
#endif

}  // namespace ee
