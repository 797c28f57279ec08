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

// Least scale the attention computes with: a smaller one of K would make the
// factor of a row and page 0, and 0 * -inf in a masked place nan; a smaller one
// of V would make its reciprocal, and the row sum, infinite.
constexpr float kScaleMin = 0x1p-64f;
constexpr float kSmScaleMin = 0x1p-32f;   // least softmax scale, for the same reason

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

// A query row as two e4m3 parts under a power of two s, the smallest with |q| <=
// 448 s: hi = e4m3(q / s), lo = e4m3(lo_factor (q / s - hi)). Eight lanes a row
// (whole warp; lanes 8 r .. 8 r + 7), 16 bf16 values each.
struct QuerySplit {
  uint4 hi, lo;
  float scale;   // s; nan where the row holds inf or nan, as the product itself would be (inf - inf)

  __device__ __forceinline__ void split(const uint4& a, const uint4& b, int lane, float lo_factor) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float x[16];
    float amax = 0.f;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float m = fabsf(x[j]);
      odd = odd || !(m < INFINITY);
      amax = fmaxf(amax, m);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const unsigned votes = __ballot_sync(0xffffffffu, odd);
    odd = (votes >> (lane & 24)) & 0xffu;
    const int e = scale_exp(amax, kScaleExpMaxK);
    const float inv = pow2f(-e);
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = x[4 * k + j] * inv;
      h[k] = e4m3x4(y[0], y[1], y[2], y[3]);
      const float2 h0 = f16x2_to_f32x2(e4m3x2_to_f16x2(h[k] & 0xffffu));
      const float2 h1 = f16x2_to_f32x2(e4m3x2_to_f16x2(h[k] >> 16));
      l[k] = e4m3x4((y[0] - h0.x) * lo_factor, (y[1] - h0.y) * lo_factor, (y[2] - h1.x) * lo_factor,
                    (y[3] - h1.y) * lo_factor);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
    scale = odd ? __int_as_float(0x7fffffff) : pow2f(e);
  }
};

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

// The issuing warp runs its loops whole, with one lane elected for the products
// themselves: in a branch of one lane every operand would be moved to the
// uniform registers that tcgen05.mma reads, for each of a tile's products anew.
// For the same reason descriptors are built as a low word (address, leading
// offset), stepped by an addition, and a constant high word (stride, version,
// 128-byte swizzle). (One lane and whole descriptors: the issuing thread alone
// took 2,900 of a tile's 3,400 cycles, of which the products need 1,450.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);
}
constexpr uint32_t kSdescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // 8-row atoms 1 KB apart, 128B swizzle

// D(tmem) (+)= A(smem) * B(smem), 8-bit operands, 32 values of k a step; by the
// elected lane.
__device__ __forceinline__ void mma_ss_f8(uint32_t leader, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%2, %6};\n\t"
      "mov.b64 b, {%3, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%1], a, b, %4, p;\n\t}\n" ::"r"(leader),
      "r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kSdescHi)
      : "memory");
}
// D(tmem) (+)= A(tmem, fp16) * B(smem, fp16), 16 values of k a step.
__device__ __forceinline__ void mma_ts_f16(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%3, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %4, p;\n\t}\n" ::"r"(leader),
      "r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kSdescHi)
      : "memory");
}
__device__ __forceinline__ void tc_commit_by(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}\n" ::"r"(leader),
      "r"(smem_u32(bar))
      : "memory");
}
// Instruction descriptor for kind::f8f6f4 with e4m3 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N, uint32_t a_mn_major,
                                                      uint32_t b_mn_major) {
  return (1u << 4) | (a_mn_major << 15) | (b_mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// A role whose wait gave up tells the others of its CTA.
template <typename Ctrl>
__device__ __forceinline__ void raise_abort(Ctrl* c, int32_t* err) {
  if (!c->abort) {
    atomicOr(err, kDevErrTimeout);
    c->abort = 1;
  }
}
// Wait bounded by time only (teardown after an abort).
__device__ __forceinline__ void wait_quiet(uint64_t* bar, uint32_t parity) {
  int zero = 0;
  mbar_wait(bar, parity, &zero);
}

constexpr int kTile8 = kBN * kHeadDim;       // a K or V tile of codes of the decode kernel: 128 rows of 128 B
constexpr int kFwdPages = 5;                 // pages of a key tile of the prompt kernel
constexpr int kPageBytes8 = kPage * kHeadDim;

// What the combine has to merge behind CTA c's first piece (attention kernel ->
// combine): the unit's rows and the CTAs that hold its pieces.
struct Kv8Cut {
  int32_t n_tok;        // query tokens of the unit, 0: nothing begins or goes on here
  int32_t tok0;         // first of them (row of o)
  int32_t head0;        // first query head
  int32_t c0, c1;       // pieces: slot 2 c0 + 1, then slots 2 (c0 + 1) .. 2 c1
  int32_t pad[3];
};

struct Kv8Params {
  BatchDev batch;
  int32_t num_pages, num_kv_heads, num_q_heads, group, layer;
  int32_t toks_per_block;          // query tokens of a work unit
  int32_t item_rows;               // rows of a partial slot
  int32_t decode;                  // the kernel for at most 16 rows
  int32_t split_tiles;             // key tiles of a piece, 0: equal stretches
  int32_t grid;                    // CTAs of the attention kernel
  int32_t causal;
  float scale_log2;
  const float* k_scale;
  const float* v_scale;
  const __nv_bfloat16* q;
  uint8_t* qs;                     // split queries [total_q][H_q][hi 128 B, lo 128 B]
  float* qscale;                   // [total_q][H_q]
  __nv_bfloat16* o;
  float* row_lse;
  float* part;                     // 2 partial slots per CTA; null: no unit is cut
  Kv8Cut* cuts;                    // [grid]
  int32_t* err;
};

// Work decomposition. A unit is (request, KV head, block of query tokens); its
// key tiles are the request's pages in groups of 8 (decode) or 5. All units lie on one line,
// request by request, and each CTA takes a stretch of it. Two measures of the
// line:
//   stretches  a unit weighs the time of its tiles and every CTA takes an equal
//              weight, whatever the requests' lengths: it holds any number of
//              whole units, whose output rows the CTA writes itself, and at
//              most two cut ones, whose partial rows go to the CTA's two slots
//              (dealing out equal splits of every unit left the busiest SM with
//              1.65 times the average work on 16 ragged requests)
//   pieces     a unit weighs its pieces of split_tiles tiles at most, and a CTA
//              takes one (any number when no unit is cut): with few units no
//              CTA pays for the start and end of two. If the pieces turn out to
//              be more than the CTAs, stretches are used after all.
// One warp of a CTA walks the stretch and hands the items to the others
// through a ring in shared memory.
// weight of a key tile with two Q tiles and with one: 5 to 4 by measurement (16
// prompts 140 us when it was set; 142 at 4 to 3, 149 at 5 to 3, 157 at 2 to 1)
constexpr int kCost2 = 5, kCost1 = 4;
constexpr int kMinWork = 2 * kCost2;       // least stretch of a CTA: two tiles
constexpr int kMinWorkDecode = 2;
constexpr int kReqCache = 16;              // requests whose geometry stays in shared memory
constexpr int kItemSlots = 4;

struct Kv8Item {
  int32_t n;            // key tiles, 0: no more items
  int32_t t_begin;
  int32_t g, rb;
  int32_t slot;         // partial slot, -1: the unit is whole
  int32_t q0, n_q, n_doc;
};

struct Kv8Ring {
  uint64_t full[kItemSlots], empty[kItemSlots];
  Kv8Item item[kItemSlots];
  int32_t total, stretch, pieces;   // the line: weight, a CTA's share of it, 1: measured in pieces
  ReqInfo req[kReqCache];
};

// The walk's code runs cold in every launch, before the first load of a page,
// so it is kept short: the kernel for at most 16 rows has one block a request
// by construction, and no loop is unrolled. (With the block count and tile size
// of both kernels in one code a decode step's first item came 2.8 us after the
// line was known.)
template <bool kDecode>
__device__ __forceinline__ int kv8_blocks(const Kv8Params& p, const ReqInfo& r) {
  if (r.n_q <= 0 || !req_ok(p.batch, r)) return 0;
  return kDecode ? 1 : ceil_div(r.n_q, p.toks_per_block);
}
__host__ __device__ constexpr int kv8_tile_pages(int decode) { return decode ? kPagesPerTile : kFwdPages; }
// Key tiles of block rb, at least one (a request without pages writes its zeros
// from a fully masked tile). Causal: the pages behind the block's last visible
// key are left out; a page holds at most 16 of the tokens that lie behind it,
// so floor(tokens / 16) whole pages do.
template <bool kDecode>
__device__ __forceinline__ int kv8_tiles(const Kv8Params& p, const ReqInfo& r, int rb) {
  int pages = r.n_pages;
  if (p.causal) {
    const int behind = kDecode ? 0 : max(r.n_q - (rb + 1) * p.toks_per_block, 0);
    pages -= min(behind, r.n_doc) / kPage;
  }
  return max(1, ceil_div(pages, kv8_tile_pages(kDecode)));
}
template <bool kDecode>
__device__ __forceinline__ int kv8_cost(const Kv8Params& p, const ReqInfo& r, int rb) {
  if (kDecode) return 1;
  return r.n_q - rb * p.toks_per_block > p.toks_per_block / kQTiles ? kCost2 : kCost1;
}
template <bool kDecode>
__device__ __forceinline__ int kv8_weight(const Kv8Params& p, const ReqInfo& r, int rb, bool pieces) {
  const int n = kv8_tiles<kDecode>(p, r, rb);
  return pieces ? ceil_div(n, p.split_tiles) : n * kv8_cost<kDecode>(p, r, rb);
}
// Weight of one KV head of a request.
template <bool kDecode>
__device__ __forceinline__ int kv8_head_work(const Kv8Params& p, const ReqInfo& r, bool pieces) {
  const int n = kv8_blocks<kDecode>(p, r);
  if (kDecode) return n ? kv8_weight<kDecode>(p, r, 0, pieces) : 0;
  int w = 0;
#pragma unroll 1
  for (int rb = 0; rb < n; ++rb) w += kv8_weight<kDecode>(p, r, rb, pieces);
  return w;
}
__device__ __forceinline__ ReqInfo kv8_req(const Kv8Params& p, const Kv8Ring* ring, int b) {
  return b < kReqCache ? ring->req[b] : load_req(p.batch, b);
}

// The line of the batch (one warp): each request's weight as an exclusive
// prefix, the total, a CTA's stretch.
template <bool kDecode>
__device__ __forceinline__ void kv8_line(const Kv8Params& p, int32_t* prefix, Kv8Ring* ring, int lane) {
  const int B = p.batch.num_requests;
  const bool one_piece_each = p.part != nullptr;   // cut units: one piece a CTA
  bool pieces = p.split_tiles > 0;
  // the first 32 requests stay in registers between the two rounds
  ReqInfo mine = {};
  if (lane < B) {
    mine = load_req(p.batch, lane);
    if (lane < kReqCache) ring->req[lane] = mine;
  }
  int64_t carry = 0;   // 31 bits for every batch that agrees with its host totals
  for (;;) {
    carry = 0;
#pragma unroll 1
    for (int base = 0; base < B; base += 32) {
      const int b = base + lane;
      int64_t cnt = 0;
      if (b < B) {
        if (base > 0) mine = load_req(p.batch, b);
        if (!req_ok(p.batch, mine) && blockIdx.x == 0) atomicOr(p.err, kDevErrGeometry);
        cnt = int64_t(p.num_kv_heads) * kv8_head_work<kDecode>(p, mine, pieces);
      }
      int64_t incl = cnt;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (b < B) prefix[b] = int(carry + incl - cnt);
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (!(pieces && one_piece_each && carry > p.grid)) break;
    pieces = false;
    if (B > 32 && lane < B) mine = load_req(p.batch, lane);
  }
  __syncwarp();
  if (carry > INT32_MAX) {
    if (lane == 0 && blockIdx.x == 0) atomicOr(p.err, kDevErrGeometry);
    for (int b = lane; b < B; b += 32) prefix[b] = 0;
    carry = 0;
  }
  if (lane == 0) {
    const int W = int(carry);
    prefix[B] = W;
    ring->total = W;
    ring->stretch = max(int((uint32_t(W) + p.grid - 1) / p.grid), pieces ? 1 : kDecode ? kMinWorkDecode : kMinWork);
    ring->pieces = pieces ? 1 : 0;
  }
  __syncwarp();
}

// The items of one CTA in order (warp-uniform).
template <bool kDecode>
struct Kv8Walk {
  int pos, end, b, per_head;
  ReqInfo req;
  Kv8Cut cut;

  __device__ __forceinline__ void start(const Kv8Ring* ring) {
    const uint32_t W = ring->total, L = ring->stretch, c = blockIdx.x;
    pos = end = 0;
    b = -1;
    per_head = 1;
    cut = {};
    if (c * uint64_t(L) >= W) return;
    pos = int(c * L);
    end = int(min(W, c * L + L));
  }
  __device__ __forceinline__ bool next(const Kv8Params& p, const int32_t* prefix, const Kv8Ring* ring, Kv8Item& it) {
    const bool pieces = ring->pieces != 0;
    while (pos < end) {
      if (b < 0 || prefix[b + 1] <= pos) {
        int lo = b < 0 ? 0 : b + 1, hi = p.batch.num_requests - 1;
#pragma unroll 1
        while (lo < hi) {  // last request with prefix <= pos
          const int mid = (lo + hi + 1) >> 1;
          if (prefix[mid] <= pos) lo = mid; else hi = mid - 1;
        }
        b = lo;
        req = kv8_req(p, ring, b);
        per_head = kv8_head_work<kDecode>(p, req, pieces);
      }
      int rem = pos - prefix[b];
      it.g = rem / per_head;
      rem -= it.g * per_head;
      it.rb = 0;
      int w = per_head;
      if (!kDecode) {
        w = kv8_weight<kDecode>(p, req, 0, pieces);
#pragma unroll 1
        while (rem >= w) {
          rem -= w;
          w = kv8_weight<kDecode>(p, req, ++it.rb, pieces);
        }
      }
      const int s = pos - rem, n = kv8_tiles<kDecode>(p, req, it.rb), cost = kv8_cost<kDecode>(p, req, it.rb);
      int t_begin, t_end;
      if (pieces) {
        const int q = n / w, r = n % w;           // piece i: q tiles, the first r pieces one more
        t_begin = rem * q + min(rem, r);
        t_end = t_begin + q + (rem < r ? 1 : 0);
        pos += 1;
      } else {
        t_begin = ceil_div(rem, cost);
        t_end = min(n, ceil_div(end - s, cost));
        pos = s + w;
      }
      if (t_begin >= t_end) continue;   // the stretch ends or begins inside the last tile
      const int cta = int(blockIdx.x);
      it.slot = t_begin > 0 ? 2 * cta : t_end < n ? 2 * cta + 1 : -1;
      it.t_begin = t_begin;
      it.n = t_end - t_begin;
      it.q0 = req.q0;
      it.n_q = req.n_q;
      it.n_doc = req.n_doc;
      if (t_begin > 0) {
        // a piece that goes on from another CTA's: the second of its unit reports the cut
        const uint32_t L = ring->stretch, c0 = uint32_t(s) / L;
        if (cta == int(c0) + 1) {
          const int last = pieces ? s + w - 1 : s + (n - 1) * cost;   // the last piece, or tile, begins here
          cut.n_tok = min(p.toks_per_block, req.n_q - it.rb * p.toks_per_block);
          cut.tok0 = req.q0 + it.rb * p.toks_per_block;
          cut.head0 = it.g * p.group;
          cut.c0 = int(c0);
          cut.c1 = int(uint32_t(last) / L);
        }
      }
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ void kv8_ring_init(Kv8Ring* ring, int readers) {
  for (int s = 0; s < kItemSlots; ++s) {
    mbar_init(&ring->full[s], 1);
    mbar_init(&ring->empty[s], readers);
  }
}
// The walking warp hands out its j-th item (n = 0: the end). False: a wait gave up.
__device__ __forceinline__ bool kv8_put(Kv8Ring* ring, uint32_t j, const Kv8Item& it, int lane, volatile int* abort) {
  const int s = j % kItemSlots;
  if (j >= kItemSlots && !mbar_wait(&ring->empty[s], (j / kItemSlots - 1) & 1, abort)) return false;
  if (lane == 0) {
    ring->item[s] = it;
    mbar_arrive(&ring->full[s]);
  }
  __syncwarp();
  return true;
}
// A reading warp takes the j-th item. False: the end, or a wait gave up (bad = 1).
__device__ __forceinline__ bool kv8_take(Kv8Ring* ring, uint32_t j, Kv8Item& it, volatile int* abort, int& bad) {
  const int s = j % kItemSlots;
  if (!mbar_wait(&ring->full[s], (j / kItemSlots) & 1, abort)) { bad = 1; return false; }
  it = ring->item[s];
  __syncwarp();   // every lane has the item before the slot is given back
  if ((threadIdx.x & 31) == 0) mbar_arrive(&ring->empty[s]);
  return it.n > 0;
}

// The pages of an item, resolved by the producer warp a window of kTiles tiles
// (up to 32 pages, one a lane) at a time: page ids run two windows ahead and
// scales one, so that no tile waits for a load. (Resolved tile by tile, with
// ids two tiles and scales one tile ahead, every tile cost a load's latency:
// 2 us a tile of 80 or of 128 keys alike.) A scale outside (0, inf), or of V
// above 128, is reported and taken as 1; one below kScaleMin counts as that.
template <int kPagesTile>
struct Kv8Pages {
  static constexpr int kTiles = 32 / kPagesTile;
  int base, next_id;          // first page reference of the item; id of this lane's page in the next window to resolve
  PageRef cur, nxt;
  float cur_k, cur_v, nxt_k, nxt_v;

  __device__ __forceinline__ int ref(int window, int lane) const {
    return base + window * (kTiles * kPagesTile) + lane;
  }
  __device__ __forceinline__ int id(const Kv8Params& p, const ReqInfo& r, int window, int lane) const {
    return lane < kTiles * kPagesTile ? load_page_id(p.batch, r, ref(window, lane)) : -1;
  }
  __device__ __forceinline__ PageRef resolve(const Kv8Params& p, const ReqInfo& r, const ChunkCache* cc, int window,
                                             int id, int lane) const {
    PageRef pg;
    pg.page = -1; pg.nvalid = 0; pg.lstart = 0; pg.chunk = -1;
    if (lane < kTiles * kPagesTile) pg = page_ref_cached(cc, p.batch, r, ref(window, lane), id, p.num_pages, p.err);
    return pg;
  }
  __device__ __forceinline__ void scales(const Kv8Params& p, const PageRef& pg, int g, float& k, float& v) const {
    k = v = 1.f;
    if (pg.page < 0 || pg.nvalid <= 0) return;
    const int64_t at = (int64_t(p.layer) * p.num_pages + pg.page) * p.num_kv_heads + g;
    k = __ldg(p.k_scale + at);
    v = __ldg(p.v_scale + at);
  }
  __device__ __forceinline__ void settle(const Kv8Params& p) {
    if (!(cur_k >= kScaleMin && cur_k < INFINITY)) {
      if (cur_k > 0.f && cur_k < 1.f) {
        cur_k = kScaleMin;
      } else {
        atomicOr(p.err, kDevErrRange);
        cur_k = 1.f;
      }
    }
    if (!(cur_v >= kScaleMin && cur_v <= 128.f)) {
      if (cur_v > 0.f && cur_v < 1.f) {
        cur_v = kScaleMin;
      } else {
        atomicOr(p.err, kDevErrRange);
        cur_v = 1.f;
      }
    }
  }
  // The first window; the next one's ids are on their way.
  __device__ __forceinline__ void start(const Kv8Params& p, const ReqInfo& r, ChunkCache* cc, bool load_chunks,
                                        int t_begin, int g, int lane) {
    base = t_begin * kPagesTile;
    const int id0 = id(p, r, 0, lane);
    next_id = id(p, r, 1, lane);
    if (load_chunks) {
      __syncwarp();
      load_chunk_cache(cc, p.batch, r, lane);
    }
    cur = resolve(p, r, cc, 0, id0, lane);
    scales(p, cur, g, cur_k, cur_v);
  }
  // Once the boxes of the first tile of a window are under way: the window after it.
  __device__ __forceinline__ void ahead(const Kv8Params& p, const ReqInfo& r, const ChunkCache* cc, int i, int g,
                                        int lane) {
    const int w = i / kTiles;
    nxt = resolve(p, r, cc, w + 1, next_id, lane);
    scales(p, nxt, g, nxt_k, nxt_v);
    next_id = id(p, r, w + 2, lane);
  }
  // The first tile of a later window.
  __device__ __forceinline__ void advance() {
    cur = nxt;
    cur_k = nxt_k;
    cur_v = nxt_v;
  }
};

cudaError_t launch_kv8_split_q(const Kv8Params&, cudaStream_t);
cudaError_t launch_kv8_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p,
                           int grid, cudaStream_t stream);
// query blocks of at most 16 rows
cudaError_t launch_kv8_decode(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p, int grid,
                              cudaStream_t stream);
cudaError_t launch_kv8_combine(const Kv8Params& p, cudaStream_t stream);

}  // namespace rag
