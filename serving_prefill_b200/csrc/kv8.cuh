// Parameter blocks, e4m3 helpers and launchers of the cache-append kernels
// and of the attention over the 8-bit pool.
//
// The 8-bit pool keeps K and V as e4m3 codes [layers][pages][H_kv][16][128]
// with one fp32 scale per (layer, page, KV head) for each of them; a value is
// code * scale. The append kernel writes powers of two as scales.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace rag {

constexpr float kE4m3Max = 448.f;
constexpr int kScaleExpMin = -24;     // smallest block scale the append writes: 2^-24
constexpr int kScaleExpMaxK = 120;    // 448 * 2^120 is past the fp32 range
constexpr int kScaleExpMaxV = 7;      // 448 * 2^7 = 57,344: V enters its product as fp16

// Two fp32 values to two e4m3 codes (lo in the low byte), nearest even,
// saturated at +-448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Two codes (low 16 bits of w) to two fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(w)));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Exponent e of the smallest 2^e with amax <= 448 * 2^e, within [kScaleExpMin, top].
// 448 = 1.75 * 2^8: the mantissa decides between exponent(amax) - 8 and - 7.
__device__ __forceinline__ int scale_exp(float amax, int top) {
  const uint32_t b = __float_as_uint(amax);
  int e = int(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < kScaleExpMin ? kScaleExpMin : e;
  return e > top ? top : e;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Tokens appended by one call: sequence s takes rows [tok_off[s], tok_off[s+1])
// of k, v and q as its tokens start[s], start[s] + 1, ...
struct AppendSeqs {
  const int32_t* tok_off;    // [n_seqs + 1]
  const int32_t* start;      // [n_seqs]
  const int32_t* page_off;   // [n_seqs + 1]
  const int32_t* page_ids;   // [total_pages]
  const int32_t* pos0;       // [n_seqs] or null: rotary position of the sequence's first token
  int32_t n_seqs, total_new, total_pages;
};
struct AppendParams {
  AppendSeqs seqs;
  uint8_t* pool_k;
  uint8_t* pool_v;
  float* k_scale;            // 8-bit pool only
  float* v_scale;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* q;          // or null
  uint8_t* q_out;
  int64_t k_stride, v_stride, q_stride;   // bytes from one token's row to the next
  const float2* rope;        // [n_pos][head_dim / 2] (cos, sin) or null
  int32_t* err;
  int32_t n_pos, layer, num_pages, num_kv_heads, num_q_heads, head_dim;
  int32_t tokens_per_block, units_per_block;   // at most 8
  int32_t heads_split;       // blocks that share a group of units
  int32_t kv_blocks;         // 8-bit pool: blocks that store K and V (the rest rotate q)
};

cudaError_t launch_kv_append(const AppendParams&, int is_f32, int grid, cudaStream_t);
cudaError_t launch_kv8_append(const AppendParams&, int grid, cudaStream_t);
cudaError_t launch_kv8_append_stream(const AppendParams&, int grid, cudaStream_t);
cudaError_t launch_rope_q(const AppendParams&, int grid, cudaStream_t);
cudaError_t launch_rope_cos_sin(double base, int head_dim, int n_pos, float2* table, cudaStream_t);

// ------------------------------------------------------------ attention

// D(tmem) (+)= A(smem desc) * B(smem desc), 8-bit operands, 32 values of k a step.
__device__ __forceinline__ void mma_ss_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor for kind::f8f6f4 with e4m3 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N, uint32_t a_mn_major,
                                                      uint32_t b_mn_major) {
  return (1u << 4) | (a_mn_major << 15) | (b_mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

constexpr int kTile8 = kBN * kHeadDim;       // a K or V tile of codes: 128 rows of 128 B
constexpr int kPageBytes8 = kPage * kHeadDim;

struct Kv8Params {
  BatchDev batch;
  int32_t num_pages, num_kv_heads, num_q_heads, group, layer;
  int32_t tiles_per_split;
  int32_t toks_per_block;          // query tokens of a work unit
  int32_t item_rows;               // partial rows an item owns
  int32_t direct;                  // 1: a unit is one item, which writes the output rows itself
  int32_t causal;
  float scale_log2;
  const float* k_scale;
  const float* v_scale;
  const __nv_bfloat16* q;
  uint8_t* qs;                     // split queries [total_q][H_q][hi 128 B, lo 128 B]
  float* qscale;                   // [total_q][H_q]
  __nv_bfloat16* o;
  float* row_lse;
  float* part;
  int32_t* item_prefix;
  int32_t* err;
  int64_t max_items;
};

// Units of a request: blocks of query tokens and splits of the key tiles.
// Every key comes from the pool, so the tiles are the request's pages alone; a
// request without pages still has one (empty) item, which writes its zeros.
__device__ __forceinline__ FwdShape kv8_shape(const Kv8Params& p, const ReqInfo& r) {
  FwdShape s;
  if (r.n_q <= 0 || !req_ok(p.batch, r)) { s.n_rt = 0; s.n_split = 0; return s; }
  s.n_rt = ceil_div(r.n_q, p.toks_per_block);
  s.n_split = max(1, ceil_div(doc_tiles(r), p.tiles_per_split));
  return s;
}

// Key tiles that hold the request's positions 0 .. last_pos.
__device__ __forceinline__ int tiles_upto(const BatchDev& B, const ReqInfo& r, int last_pos) {
  const int all = doc_tiles(r);
  if (last_pos >= r.n_doc - 1) return all;
  if (last_pos < 0) return 0;
  int lo = r.c0, hi = r.c1 - 1;   // last chunk that starts at or before last_pos
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(B.chunk_doc_off + mid) - r.doc0 <= last_pos) lo = mid; else hi = mid - 1;
  }
  const int page = __ldg(B.chunk_page_off + lo) - r.p0 + (last_pos - (__ldg(B.chunk_doc_off + lo) - r.doc0)) / kPage;
  return page < 0 ? all : min(all, page / kPagesPerTile + 1);
}

struct Kv8Item {
  int b, g, rb, split;
  int t_begin, t_end;
  ReqInfo req;
};

__device__ __forceinline__ Kv8Item kv8_item(const Kv8Params& p, const int32_t* prefix, int w) {
  int lo = 0, hi = p.batch.num_requests - 1;
  while (lo < hi) {  // last b with prefix[b] <= w
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= w) lo = mid; else hi = mid - 1;
  }
  Kv8Item it;
  it.b = lo;
  it.req = load_req(p.batch, lo);
  const FwdShape sh = kv8_shape(p, it.req);
  int local = w - prefix[lo];
  it.rb = local % sh.n_rt;
  local /= sh.n_rt;
  it.split = local % sh.n_split;
  it.g = local / sh.n_split;
  int n_tiles = doc_tiles(it.req);
  if (p.causal && it.rb < sh.n_rt - 1)
    n_tiles = tiles_upto(p.batch, it.req, it.req.n_doc - it.req.n_q + (it.rb + 1) * p.toks_per_block - 1);
  it.t_begin = min(it.split * p.tiles_per_split, n_tiles);
  it.t_end = min(it.t_begin + p.tiles_per_split, n_tiles);
  return it;
}

// Items of every request as an exclusive prefix in shared memory (one warp).
// Returns the total, 0 (reported) when it exceeds what the workspace holds.
__device__ __forceinline__ int kv8_prefix(const Kv8Params& p, int32_t* prefix, int lane) {
  const int B = p.batch.num_requests;
  int carry = 0;
  for (int base = 0; base < B; base += 32) {
    const int b = base + lane;
    int cnt = 0;
    if (b < B) {
      const ReqInfo r = load_req(p.batch, b);
      if (!req_ok(p.batch, r) && blockIdx.x == 0) atomicOr(p.err, kDevErrGeometry);
      const FwdShape sh = kv8_shape(p, r);
      cnt = p.num_kv_heads * sh.n_split * sh.n_rt;
    }
    int incl = cnt;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (b < B) prefix[b] = carry + incl - cnt;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
  if (carry > p.max_items) {
    if (blockIdx.x == 0 && lane == 0) atomicOr(p.err, kDevErrGeometry);
    carry = 0;
    for (int b = lane; b < B; b += 32) prefix[b] = 0;
  }
  if (lane == 0) prefix[B] = carry;
  return carry;
}

// The page that lane `lane & 7` of a producer warp loads for a tile, and its
// scale (lanes 0-7: K's, lanes 8-15: V's). A scale outside (0, inf), or of V
// above 128, is reported and taken as 1.
struct PageScale {
  PageRef pg;
  float scale;
};
__device__ __forceinline__ float page_scale_load(const Kv8Params& p, const PageRef& pg, int g, int lane) {
  if (pg.page < 0 || pg.nvalid <= 0 || lane >= 16) return 1.f;
  const float* at = (lane < 8 ? p.k_scale : p.v_scale) + (int64_t(p.layer) * p.num_pages + pg.page) * p.num_kv_heads + g;
  return __ldg(at);
}
__device__ __forceinline__ float page_scale_ok(const Kv8Params& p, float s, int lane) {
  if (s > 0.f && s <= (lane < 8 ? 3.3e38f : 128.f)) return s;
  atomicOr(p.err, kDevErrRange);
  return 1.f;
}

cudaError_t launch_kv8_split_q(const Kv8Params&, cudaStream_t);
cudaError_t launch_kv8_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p,
                           int grid, cudaStream_t stream);
// query blocks of at most 16 rows
cudaError_t launch_kv8_decode(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p, int grid,
                              cudaStream_t stream);
cudaError_t launch_kv8_combine(const Kv8Params& p, int max_q, cudaStream_t stream);

}  // namespace rag
