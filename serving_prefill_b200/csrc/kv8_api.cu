// Host side of the cache-append entry points and of the attention over the
// 8-bit pool: argument validation, work planning and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "rag_prefill.h"
#include "host.cuh"
#include "kv8.cuh"

namespace rag {

constexpr int kMaxAppendSeqs = 65536;

static rag_status check_pool8(const rag_kv8_pool* pool) {
  if (!pool || !pool->k || !pool->v || !pool->k_scale || !pool->v_scale) return RAG_ERR_INVALID_ARG;
  if (!aligned16(pool->k) || !aligned16(pool->v)) return RAG_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(pool->k_scale) | reinterpret_cast<uintptr_t>(pool->v_scale)) & 3u)
    return RAG_ERR_INVALID_ARG;
  if (pool->page_size != kPage || pool->head_dim != kHeadDim) return RAG_ERR_UNSUPPORTED;
  if (pool->num_layers <= 0 || pool->num_pages <= 0 || pool->num_kv_heads <= 0) return RAG_ERR_SHAPE;
  const int64_t rows = int64_t(pool->num_layers) * pool->num_pages * pool->num_kv_heads;
  if (rows >= (int64_t(1) << 27)) return RAG_ERR_UNSUPPORTED;   // 2^31 rows of 16 slots
  return RAG_OK;
}

// What the append entry points share; fills everything but the pool's pointers.
static rag_status check_append(AppendParams& p, int elem, int num_layers, int layer, const rag_append* seqs,
                               const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* rope,
                               int32_t n_pos, const void* q, int64_t q_stride, int32_t num_q_heads, void* q_out,
                               int32_t* device_err) {
  if (!seqs || layer < 0 || layer >= num_layers) return RAG_ERR_INVALID_ARG;
  if (seqs->n_seqs < 0 || seqs->total_new < 0 || seqs->total_pages < 0) return RAG_ERR_SHAPE;
  if (seqs->n_seqs > kMaxAppendSeqs) return RAG_ERR_UNSUPPORTED;
  if (seqs->n_seqs == 0 || seqs->total_new == 0) return RAG_OK;
  if (!seqs->tok_off || !seqs->start || !seqs->page_off || !seqs->page_ids || !k || !v) return RAG_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return RAG_ERR_INVALID_ARG;
  if (rope && n_pos <= 0) return RAG_ERR_INVALID_ARG;
  if (q && num_q_heads <= 0) return RAG_ERR_SHAPE;
  const int64_t kv_row = int64_t(p.num_kv_heads) * p.head_dim;
  const int64_t q_row = int64_t(num_q_heads) * p.head_dim;
  if (k_stride < kv_row || v_stride < kv_row || (q && q_stride < q_row)) return RAG_ERR_SHAPE;
  if (q == q_out && q && q_stride != q_row) return RAG_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(rope) ||
      (k_stride * elem) % 16 || (v_stride * elem) % 16 || (q && (q_stride * elem) % 16))
    return RAG_ERR_INVALID_ARG;
  p.seqs.tok_off = seqs->tok_off;
  p.seqs.start = seqs->start;
  p.seqs.page_off = seqs->page_off;
  p.seqs.page_ids = seqs->page_ids;
  p.seqs.pos0 = seqs->pos0;
  p.seqs.n_seqs = seqs->n_seqs;
  p.seqs.total_new = seqs->total_new;
  p.seqs.total_pages = seqs->total_pages;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.q = static_cast<const uint8_t*>(q);
  p.q_out = static_cast<uint8_t*>(q_out);
  p.k_stride = k_stride * elem;
  p.v_stride = v_stride * elem;
  p.q_stride = q ? q_stride * elem : 0;
  p.rope = reinterpret_cast<const float2*>(rope);
  p.err = device_err;
  p.n_pos = rope ? n_pos : 0;
  p.layer = layer;
  p.num_q_heads = q ? num_q_heads : 0;
  // enough blocks to fill the GPU twice before a block takes several tokens
  p.tokens_per_block = std::max(1, std::min(8, seqs->total_new / (4 * num_sms())));
  p.kv_blocks = 0;
  return RAG_OK;
}

}  // namespace rag

using namespace rag;

extern "C" {

rag_status rag_rope_cos_sin(double base, int32_t head_dim, int32_t n_pos, float* table, void* stream) {
  if (!(base > 1.0) || !std::isfinite(base) || !table || !aligned16(table) || n_pos < 0) return RAG_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return RAG_ERR_UNSUPPORTED;
  if (n_pos == 0) return RAG_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope ls(kKindRopeTable, s);
  cudaError_t e = launch_rope_cos_sin(base, head_dim, n_pos, reinterpret_cast<float2*>(table), s);
  ls.done(e);
  return e == cudaSuccess ? RAG_OK : RAG_ERR_CUDA;
}

rag_status rag_kv_append(const rag_kv_pool* pool, int32_t layer, const rag_append* seqs, const void* k,
                         int64_t k_stride, const void* v, int64_t v_stride, const float* rope, int32_t n_pos,
                         const void* q, int64_t q_stride, int32_t num_q_heads, void* q_out, int32_t* device_err,
                         void* stream) {
  rag_status st = check_pool(pool);
  if (st != RAG_OK) return st;
  const bool f32 = pool->dtype == RAG_F32;
  AppendParams p = {};
  p.num_kv_heads = pool->num_kv_heads;
  p.num_pages = pool->num_pages;
  p.head_dim = pool->head_dim;
  st = check_append(p, f32 ? 4 : 2, pool->num_layers, layer, seqs, k, k_stride, v, v_stride, rope, n_pos, q, q_stride,
                    num_q_heads, q_out, device_err);
  if (st != RAG_OK || seqs->n_seqs == 0 || seqs->total_new == 0) return st;
  p.pool_k = static_cast<uint8_t*>(pool->k);
  p.pool_v = static_cast<uint8_t*>(pool->v);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope ls(kKindKvAppend, s);
  cudaError_t e = launch_kv_append(p, f32, cdiv(seqs->total_new, p.tokens_per_block), s);
  ls.done(e);
  return e == cudaSuccess ? RAG_OK : RAG_ERR_CUDA;
}

rag_status rag_kv8_append(const rag_kv8_pool* pool, int32_t layer, const rag_append* seqs, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, const float* rope, int32_t n_pos,
                          const void* q, int64_t q_stride, int32_t num_q_heads, void* q_out, int32_t* device_err,
                          void* stream) {
  rag_status st = check_pool8(pool);
  if (st != RAG_OK) return st;
  AppendParams p = {};
  p.num_kv_heads = pool->num_kv_heads;
  p.num_pages = pool->num_pages;
  p.head_dim = pool->head_dim;
  st = check_append(p, 2, pool->num_layers, layer, seqs, k, k_stride, v, v_stride, rope, n_pos, q, q_stride,
                    num_q_heads, q_out, device_err);
  if (st != RAG_OK || seqs->n_seqs == 0 || seqs->total_new == 0) return st;
  p.pool_k = static_cast<uint8_t*>(pool->k);
  p.pool_v = static_cast<uint8_t*>(pool->v);
  p.k_scale = pool->k_scale;
  p.v_scale = pool->v_scale;
  // units of a call: see kv8_append_kernel
  const int64_t units = int64_t(seqs->total_new) / kPage + 2 * int64_t(seqs->n_seqs);
  const int64_t kv_blocks = (units * 2 * p.num_kv_heads + 7) / 8;
  const int64_t q_blocks = q ? cdiv(seqs->total_new, p.tokens_per_block) : 0;
  if (kv_blocks + q_blocks >= (int64_t(1) << 31)) return RAG_ERR_UNSUPPORTED;
  p.kv_blocks = int(kv_blocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope ls(kKindKv8Append, s);
  cudaError_t e = launch_kv8_append(p, int(kv_blocks + q_blocks), s);
  ls.done(e);
  return e == cudaSuccess ? RAG_OK : RAG_ERR_CUDA;
}

}  // extern "C"
