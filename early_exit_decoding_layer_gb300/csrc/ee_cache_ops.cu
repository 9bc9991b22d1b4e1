// C entry points of the operators on the paged cache: argument checks, all
// on the host and before any CUDA call, then one launch.
#include <algorithm>

#include "ee_cache_ops.cuh"

namespace ee {
namespace {

bool aligned(const void* p, uintptr_t a) { return p && (uintptr_t)p % a == 0; }

// The checks common to the four, and the cache they describe.
ee_status paged_cache(int32_t n_seqs, int32_t n_kv_heads, int32_t head_dim, int32_t max_ctx, const uint16_t* k,
                      const uint16_t* v, float* weights, int32_t n_blocks, const int32_t* table, int32_t stride,
                      int32_t* err, PagedCache* c) {
  if (n_seqs < 1 || n_seqs > EE_MAX_BATCH || n_kv_heads < 1 || n_kv_heads > 1024 || (head_dim != 64 && head_dim != 128))
    return EE_ERR_INVALID_ARG;
  if (max_ctx < 1 || max_ctx > kCacheMaxCtx || n_blocks < 1 || stride < 1) return EE_ERR_INVALID_ARG;
  // rows of the cache as one matrix: tensor map coordinates are 32 bits
  if ((int64_t)n_blocks * n_kv_heads * EE_KV_BLOCK > INT32_MAX) return EE_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(table, 4)) return EE_ERR_INVALID_ARG;
  c->k = k;
  c->v = v;
  c->weights = weights;
  c->table = table;
  c->table_stride = stride;
  c->n_blocks = n_blocks;
  c->n_kv_heads = n_kv_heads;
  c->head_dim = head_dim;
  c->max_ctx = (int32_t)std::min<int64_t>(max_ctx, (int64_t)stride * EE_KV_BLOCK);
  c->err = err;
  return EE_OK;
}

bool group_ok(int32_t n_heads, int32_t n_kv_heads) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads) return false;
  const int G = n_heads / n_kv_heads;
  return G == 1 || G == 2 || G == 4 || G == 8;
}

// A row stride in fp16 elements: whole 16-byte chunks, and within what a
// tensor map takes (2^40 bytes).
bool stride_ok(int64_t stride, int32_t n_heads, int32_t head_dim) {
  return stride >= (int64_t)n_heads * head_dim && stride % 8 == 0 && stride < ((int64_t)1 << 38);
}

ee_status prompt_args(int32_t n_seqs, int32_t total_q, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                      const uint16_t* q, int64_t q_stride, const int32_t* cu_q, const int32_t* ctx, PromptParams* p) {
  // 2^24 rows keep every tile count within 32 bits
  if (total_q < 0 || total_q > (1 << 24) || !group_ok(n_heads, n_kv_heads) || !stride_ok(q_stride, n_heads, head_dim))
    return EE_ERR_INVALID_ARG;
  if ((total_q > 0 && !aligned(q, 16)) || !aligned(cu_q, 4) || !aligned(ctx, 4)) return EE_ERR_INVALID_ARG;
  p->n_seqs = n_seqs;
  p->total_q = total_q;
  p->n_heads = n_heads;
  p->q = q;
  p->q_stride = q_stride;
  p->cu_q = cu_q;
  p->ctx = ctx;
  return EE_OK;
}

ee_status launched(cudaError_t e) {
  if (e == cudaSuccess) return EE_OK;
  cudaGetLastError();  // reported by the status, not to a later call
  return EE_ERR_CUDA;
}

}  // namespace
}  // namespace ee

using namespace ee;

extern "C" {

ee_status ee_op_prompt_attention(int32_t n_seqs, int32_t total_q, int32_t n_heads, int32_t n_kv_heads,
                                 int32_t head_dim, int32_t max_ctx, const uint16_t* q, int64_t q_stride,
                                 const uint16_t* kcache, const uint16_t* vcache, int32_t n_blocks,
                                 const int32_t* block_table, int32_t bt_stride, const int32_t* cu_q,
                                 const int32_t* ctx, uint16_t* o, int64_t o_stride, float* lse, int32_t* err_flag,
                                 void* stream) {
  PromptParams p;
  ee_status s = paged_cache(n_seqs, n_kv_heads, head_dim, max_ctx, kcache, vcache, nullptr, n_blocks, block_table,
                            bt_stride, err_flag, &p.c);
  if (s == EE_OK) s = prompt_args(n_seqs, total_q, n_heads, n_kv_heads, head_dim, q, q_stride, cu_q, ctx, &p);
  if (s != EE_OK) return s;
  if (!aligned(vcache, 16) || !stride_ok(o_stride, n_heads, head_dim) || (lse && !aligned(lse, 4)))
    return EE_ERR_INVALID_ARG;
  if (total_q == 0) return EE_OK;
  if (!aligned(o, 16)) return EE_ERR_INVALID_ARG;
  // columns of one allocation may interleave q and o; equal starts may not
  if (o == q) return EE_ERR_INVALID_ARG;
  p.o = o;
  p.o_stride = o_stride;
  p.lse = lse;
  return launched(launch_prompt_attention(p, (cudaStream_t)stream));
}

ee_status ee_op_prompt_weights(int32_t n_seqs, int32_t total_q, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                               int32_t max_ctx, const uint16_t* q, int64_t q_stride, const uint16_t* kcache,
                               int32_t n_blocks, const int32_t* block_table, int32_t bt_stride, const int32_t* cu_q,
                               const int32_t* ctx, const float* lse, float* weights, int32_t* err_flag,
                               void* stream) {
  PromptParams p;
  ee_status s = paged_cache(n_seqs, n_kv_heads, head_dim, max_ctx, kcache, nullptr, weights, n_blocks, block_table,
                            bt_stride, err_flag, &p.c);
  if (s == EE_OK) s = prompt_args(n_seqs, total_q, n_heads, n_kv_heads, head_dim, q, q_stride, cu_q, ctx, &p);
  if (s != EE_OK) return s;
  if (!aligned(weights, 16)) return EE_ERR_INVALID_ARG;
  if (total_q == 0) return EE_OK;
  if (!aligned(lse, 4)) return EE_ERR_INVALID_ARG;
  p.lse_in = lse;
  return launched(launch_prompt_weights(p, (cudaStream_t)stream));
}

ee_status ee_op_attention_weights(int32_t B, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_ctx,
                                  const float* q, const uint16_t* kcache, const uint16_t* vcache, int32_t n_blocks,
                                  const int32_t* block_table, int32_t bt_stride, const int32_t* pos, float* o,
                                  float* weights, int32_t* err_flag, void* stream) {
  DecodeWeightsParams p;
  const ee_status s = paged_cache(B, n_kv_heads, head_dim, max_ctx, kcache, vcache, weights, n_blocks, block_table,
                                  bt_stride, err_flag, &p.c);
  if (s != EE_OK) return s;
  if (!group_ok(n_heads, n_kv_heads) || !aligned(vcache, 16) || !aligned(weights, 16) || !aligned(q, 16) ||
      !aligned(o, 16) || !aligned(pos, 4))
    return EE_ERR_INVALID_ARG;
  p.batch = B;
  p.n_heads = n_heads;
  p.q = q;
  p.pos = pos;
  p.o = o;
  return launched(launch_attention_weights(p, (cudaStream_t)stream));
}

ee_status ee_op_evict(int32_t B, int32_t n_kv_heads, int32_t head_dim, int32_t max_ctx, int32_t keep, int32_t recent,
                      uint16_t* kcache, uint16_t* vcache, float* weights, int32_t n_blocks, const int32_t* block_table,
                      int32_t bt_stride, const int32_t* dst_table, int32_t dst_stride, const int32_t* ctx,
                      int32_t* new_ctx, int32_t* kept, int32_t* err_flag, void* stream) {
  EvictParams p;
  const ee_status s = paged_cache(B, n_kv_heads, head_dim, max_ctx, kcache, vcache, weights, n_blocks, block_table,
                                  bt_stride, err_flag, &p.c);
  if (s != EE_OK) return s;
  if (!aligned(vcache, 16) || !aligned(weights, 16) || !aligned(ctx, 4) || !aligned(new_ctx, 4) || new_ctx == ctx ||
      (kept && !aligned(kept, 4)))
    return EE_ERR_INVALID_ARG;
  if (keep < 1 || keep > kCacheMaxCtx || recent < 0 || recent > keep) return EE_ERR_INVALID_ARG;
  if (dst_table && (!aligned(dst_table, 4) || dst_stride < 1 || (int64_t)dst_stride * EE_KV_BLOCK < std::min(keep, max_ctx)))
    return EE_ERR_INVALID_ARG;
  p.batch = B;
  p.keep = keep;
  p.recent = recent;
  p.dst_table = dst_table ? dst_table : block_table;
  p.dst_stride = dst_table ? dst_stride : bt_stride;
  p.ctx = ctx;
  p.new_ctx = new_ctx;
  p.kept = kept;
  return launched(launch_evict(p, (cudaStream_t)stream));
}

}  // extern "C"
