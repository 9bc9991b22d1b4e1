// Parameters and launchers of the operators on the paged cache: attention of
// packed prompt rows, the weights of its tokens, decode attention that adds
// weights, eviction.  Lengths and block ids come from device memory and are
// checked here, in the kernels: what is out of range is cut to the range and
// reported in the error word.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
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

cudaError_t launch_prompt_attention(const PromptParams& p, cudaStream_t st);
cudaError_t launch_prompt_weights(const PromptParams& p, cudaStream_t st);
cudaError_t launch_attention_weights(const DecodeWeightsParams& p, cudaStream_t st);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t st);

#ifdef __CUDACC__
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
#endif

}  // namespace ee
