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
  int32_t tokens_per_block;
  int32_t kv_blocks;         // 8-bit pool: blocks that store K and V (the rest rotate q)
};

cudaError_t launch_kv_append(const AppendParams&, int is_f32, int grid, cudaStream_t);
cudaError_t launch_kv8_append(const AppendParams&, int grid, cudaStream_t);
cudaError_t launch_rope_cos_sin(double base, int head_dim, int n_pos, float2* table, cudaStream_t);

}  // namespace rag
