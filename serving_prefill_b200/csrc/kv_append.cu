// Append of new tokens' K and V to paged caches, with the rotary rotation of
// their positions (and of the queries) on the way. The pages' listings grow a
// cache along the sequence axis (TurboRAG page, "Technical Details", listing
// `turborag_inference`: the generation continues on the concatenated cache)
// and require one set of position ids for precompute and inference (its
// "Implementation"); these kernels are that step on the paged pool.
//
// Token t of sequence s is token i = start + t - tok_off of the sequence: it
// goes to page i / 16 of the sequence's list, slot i % 16, and carries rotary
// position pos0 + i. Rotation of pair (a, b) = (x[j], x[j + d/2]) by the
// table's (c, s): a' = a c - b s, b' = b c + a s, each product and sum rounded
// to fp32 on its own (no fused multiply-add, so that the stored value is a
// function of the formula and not of a compiler's contraction), then one
// rounding to the stored type. When a call writes slot 0 of a page it zeroes
// the slots behind its last token there, so that a page never holds what an
// earlier owner left.
//
// The work is a stream: rows of 128 (or 64) values in, the same rows out, one
// 16-byte load from each half of a row per lane, so the kernels are bound by
// HBM for many tokens and by their chain of dependent loads (sequence, page
// id) for a few.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv8.cuh"
#include "leave.cuh"
#include "params.cuh"

namespace rag {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxTokensPerBlock = 8;

struct Tok {
  int64_t off;       // byte of its slot in head 0's page block of the pool; -1: not stored
  int32_t slot;
  int32_t pos;       // row of the table; -1: outside it (the row becomes zeros)
  int32_t tail;      // slots behind this token to zero
  int32_t live;      // 0: a row behind the last sequence
};

// Last s with key(s) <= x, key rising (0 when there is none), by the whole
// warp: 32 probes a round, so that up to 32 sequences cost one load's latency
// instead of five.
template <typename Key>
__device__ __forceinline__ int last_at_or_before(int n, int x, int lane, Key key) {
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, lane * step < len && key(at) <= x);
    const int k = max(__popc(le) - 1, 0);
    len = min(step, len - k * step);
    lo += k * step;
  }
  return lo;
}

// One sequence's geometry; ok = 0 when its descriptors are inconsistent.
struct Seq {
  int32_t t0, n, start, p0, n_pages, pos0, ok;
};
__device__ __forceinline__ Seq load_seq(const AppendSeqs& a, int s) {
  Seq q;
  q.t0 = __ldg(a.tok_off + s);
  const int t1 = __ldg(a.tok_off + s + 1);
  q.start = __ldg(a.start + s);
  q.p0 = __ldg(a.page_off + s);
  const int p1 = __ldg(a.page_off + s + 1);
  q.pos0 = a.pos0 ? __ldg(a.pos0 + s) : 0;
  q.n = t1 - q.t0;
  q.n_pages = p1 - q.p0;
  q.ok = q.t0 >= 0 && q.n >= 0 && t1 <= a.total_new &&
         (q.n == 0 || (q.start >= 0 && q.p0 >= 0 && q.n_pages >= 0 && p1 <= a.total_pages &&
                       int64_t(q.start) + q.n <= min(int64_t(q.n_pages) * kPage, int64_t(INT32_MAX))));
  return q;
}

// Resolve token t (whole warp; lane 0 reports).
__device__ __forceinline__ Tok token_of(const AppendParams& p, int t, int row_bytes, int lane, bool report) {
  Tok k;
  k.off = -1; k.slot = 0; k.pos = -1; k.tail = 0; k.live = 0;
  report = report && lane == 0 && p.err;
  const int end = __ldg(p.seqs.tok_off + p.seqs.n_seqs);
  const int s = last_at_or_before(p.seqs.n_seqs, t, lane, [&](int i) { return __ldg(p.seqs.tok_off + i); });
  if (t >= p.seqs.total_new || t >= end) return k;
  k.live = 1;
  const Seq q = load_seq(p.seqs, s);
  const int at = t - q.t0;
  if (!q.ok || at < 0 || at >= q.n) {
    if (report) atomicOr(p.err, kDevErrGeometry);
    return k;
  }
  const int i = q.start + at;
  const int64_t pos = int64_t(q.pos0) + i;
  if (!p.rope) {
    k.pos = 0;
  } else if (pos >= 0 && pos < p.n_pos) {
    k.pos = int32_t(pos);
  } else if (report) {
    atomicOr(p.err, kDevErrGeometry);
  }
  const int page = __ldg(p.seqs.page_ids + q.p0 + i / kPage);
  if (page < 0 || page >= p.num_pages) {
    if (report) atomicOr(p.err, kDevErrPage);
    return k;
  }
  k.slot = i % kPage;
  k.off = ((int64_t(p.layer) * p.num_pages + page) * p.num_kv_heads * kPage + k.slot) * row_bytes;
  if (at == q.n - 1 && i - k.slot >= q.start) k.tail = kPage - 1 - k.slot;
  return k;
}

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return bits_f2(d);
}

__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// As fmax3, but a nan comes through.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two pairs turned at once (x of a and b: one pair, y: the next): a c - b s and
// b c + a s, every product and sum rounded on its own, which is part of the
// operator (see above). The scalar intrinsics are never contracted; packed
// products followed by packed sums were fused on their way to the machine.
__device__ __forceinline__ void turn2(float2& a, float2& b, float4 cs) {   // cs: both cosines, both sines
  const float ax = __fsub_rn(__fmul_rn(a.x, cs.x), __fmul_rn(b.x, cs.z));
  const float ay = __fsub_rn(__fmul_rn(a.y, cs.y), __fmul_rn(b.y, cs.w));
  b.x = __fadd_rn(__fmul_rn(b.x, cs.x), __fmul_rn(a.x, cs.z));
  b.y = __fadd_rn(__fmul_rn(b.y, cs.y), __fmul_rn(a.y, cs.w));
  a.x = ax;
  a.y = ay;
}

// A table row in shared memory: the vector (two pairs) that lane c of a row
// reads j-th lies at [j][c], so that the lanes of a row read neighbouring
// vectors; in the table they lie 16 N / 2 bytes apart, which costs a cache line
// a lane (the table's reads then took longer than the rows'). Within a vector
// the two cosines come first, as the packed products take them.
__device__ __forceinline__ float4 tab_vec(const float4* at) {
  const float4 v = __ldg(at);
  return make_float4(v.x, v.z, v.y, v.w);
}
template <int N>
__device__ __forceinline__ int tab_at(int f, int lanes) { return f % (N / 2) * lanes + f / (N / 2); }

// A row's two 16-byte vectors (one of each half) as they lie in memory.
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw load_raw(const uint8_t* at, int half_bytes) {
  Raw r;
  r.a = *reinterpret_cast<const uint4*>(at);   // not the read-only path: q may be rotated in place
  r.b = *reinterpret_cast<const uint4*>(at + half_bytes);
  return r;
}
// 16 bytes of a row as fp32 pairs, and back.
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float2* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const float2* x) {
    return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                      pack_bf16x2(x[3].x, x[3].y));
  }
};
template <> struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float2* x) {
    x[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    x[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  static __device__ __forceinline__ uint4 pack(const float2* x) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  }
};

// Rows of the tokens t0 .. t0 + n_tok - 1 of a block of tpb tokens (a power of
// two): K heads (kKV), V heads (kKV) and query heads, a group of d/2 / (16 /
// sizeof(T)) lanes a row. A group keeps to one token, so that its table vectors
// are read once and stay in registers. What a row holds does not depend on
// where it goes: the first kAhead rows of every group are requested before the
// tokens are resolved (a warp a token) and arrive under that chain of
// dependent loads.
constexpr int kAhead = 2;

template <typename T, int kDim, bool kKV>
__device__ __forceinline__ void store_rows(const AppendParams& p, Tok* toks, float4* tab, int t0, int tpb) {
  constexpr int N = Vec<T>::kN;
  constexpr int kHalf = kDim / 2, kHalfBytes = kHalf * int(sizeof(T)), kRowBytes = 2 * kHalfBytes;
  constexpr int kLanes = kHalf / N;                // lanes of one row
  constexpr int kGroups = kAppendThreads / kLanes;
  const int c = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const int H = p.num_kv_heads;
  const int kv = kKV ? 2 * H : 0;
  const int rows = kv + p.num_q_heads;             // num_q_heads is 0 without queries
  const int n_tok = min(tpb, p.seqs.total_new - t0);
  const int gpt = kGroups / tpb;                   // groups of a token
  const int n = grp / gpt, r0 = grp % gpt;
  const int64_t t = t0 + n;
  const bool mine = n < n_tok;
  Raw raw[kAhead];
  auto load = [&](Raw& w, int row) {
    if (!mine || row >= rows) return;
    const uint8_t* base = p.q;
    int64_t stride = p.q_stride;
    int r = row - kv;
    if (kKV && r < 0) {
      const bool is_k = row < H;
      base = is_k ? p.k : p.v;
      stride = is_k ? p.k_stride : p.v_stride;
      r = is_k ? row : row - H;
    }
    w = load_raw(base + t * stride + uint32_t(r * kRowBytes + c * 16), kHalfBytes);
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) load(raw[j], r0 + j * gpt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < n_tok) {
    const Tok k = token_of(p, t0 + warp, kRowBytes, lane, kKV);
    if (lane == 0) toks[warp] = k;
    if (p.rope && k.pos >= 0) {
      const float4* row = reinterpret_cast<const float4*>(p.rope + int64_t(k.pos) * kHalf);
      if (lane < kHalf / 2) tab[warp * (kHalf / 2) + tab_at<N>(lane, kLanes)] = tab_vec(row + lane);
    }
  }
  __syncthreads();
  if (!mine) return;
  const Tok k = toks[n];
  const bool zero = k.pos < 0, turning = p.rope != nullptr && !zero;
  float4 cs[N / 2];
  if (turning) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) cs[j] = tab[n * (kHalf / 2) + j * kLanes + c];
  }
  bool over = false;
  for (int row0 = r0; row0 < rows; row0 += kAhead * gpt) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int row = row0 + j * gpt;
      if (row >= rows) break;
      int r = row - kv;
      bool store = k.live, is_v = false;
      uint8_t* dst = p.q_out + t * (p.num_q_heads * kRowBytes) + uint32_t(r * kRowBytes);
      if (kKV && r < 0) {
        is_v = row >= H;
        r = is_v ? row - H : row;
        store = k.off >= 0;
        dst = (is_v ? p.pool_v : p.pool_k) + k.off + uint32_t(r * (kPage * kRowBytes));
      }
      Raw w = raw[j];
      load(raw[j], row + kAhead * gpt);
      if (!store) continue;
      if (zero) {
        w = Raw{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      } else if (turning && !is_v) {
        float2 a[N / 2], b[N / 2];
        Vec<T>::unpack(w.a, a);
        Vec<T>::unpack(w.b, b);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) turn2(a[i], b[i], cs[i]);
        w.a = Vec<T>::pack(a);
        w.b = Vec<T>::pack(b);
      }
      if (sizeof(T) == 2 && is_v) {   // V of a bf16 cache is stored as fp16 (saturated, reported)
        uint32_t range = 0;
        w.a = bf16x8_to_f16x8(w.a, range);
        w.b = bf16x8_to_f16x8(w.b, range);
        over = over || range_exceeded(range);
      }
      *reinterpret_cast<uint4*>(dst + c * 16) = w.a;
      *reinterpret_cast<uint4*>(dst + kHalfBytes + c * 16) = w.b;
    }
  }
  if (over && p.err) atomicOr(p.err, kDevErrRange);
}

}  // namespace

// A block stores tokens_per_block tokens.
template <typename T, int kDim>
__global__ void __launch_bounds__(kAppendThreads, 3) kv_append_kernel(const AppendParams p) {
  __shared__ Tok toks[kMaxTokensPerBlock];
  __shared__ float4 tab[kMaxTokensPerBlock * 32];
  const int t0 = blockIdx.x * p.tokens_per_block;
  store_rows<T, kDim, true>(p, toks, tab, t0, p.tokens_per_block);
  // slots behind a sequence's last token in a page this call began
  const int H = p.num_kv_heads;
  constexpr int row_bytes = kDim * int(sizeof(T));
  for (int n = 0; n < min(p.tokens_per_block, p.seqs.total_new - t0); ++n) {
    const Tok k = toks[n];
    if (k.off < 0 || k.tail == 0) continue;
    const int vecs = k.tail * row_bytes / 16;
    for (int x = threadIdx.x; x < 2 * H * vecs; x += kAppendThreads) {
      const int h = x / vecs % H;
      uint8_t* base = (x / vecs < H ? p.pool_k : p.pool_v) + k.off + (int64_t(h) * kPage + 1) * row_bytes;
      reinterpret_cast<uint4*>(base)[x % vecs] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

// 8-bit pool. A warp settles one (page the call touches, KV head) of K or of V
// at a time: the block scale needs the largest magnitude of all its new rows,
// and a scale that grows has to bring the page's held codes along, so the page
// block is the unit that one warp can settle alone, with no atomics. The rows
// stay in registers as they were read and are turned twice, for the maximum and
// for the codes: kept as fp32 they would take 64 registers a lane, and the
// kernel lives on warps in flight. The pages are found without a prefix kernel:
// sequence s owns the unit numbers from tok_off[s] / 16 + 2 s on, which leaves
// room for every page that its n tokens can touch ((n + 14) / 16 + 1 at most);
// units past a sequence's last page have nothing to do. A block resolves
// units_per_block units at once, a warp each (resolved by every warp for
// itself, the chain of about ten dependent loads took longer than the rows),
// and walks their page blocks with the unit's table rows in shared memory.
// Lane (r, c) = (lane / 8, lane % 8) holds columns 8c.. and 64 + 8c.. of rows
// r, r + 4, r + 8, r + 12.
namespace {

struct Unit {
  int64_t page;        // -1: nothing to do
  int32_t s0, s1;      // new slots
  int32_t t0;          // row of k and v that slot 0 would have
  int32_t pos;         // rotary position that slot 0 would have
};

__device__ __forceinline__ Unit unit_of(const AppendParams& p, int u, int lane) {
  Unit x;
  x.page = -1; x.s0 = x.s1 = x.t0 = x.pos = 0;
  const int s = last_at_or_before(p.seqs.n_seqs, u, lane,
                                  [&](int i) { return __ldg(p.seqs.tok_off + i) / kPage + 2 * i; });
  const Seq q = load_seq(p.seqs, s);
  const bool report = lane == 0 && p.err;
  if (!q.ok) {
    if (report) atomicOr(p.err, kDevErrGeometry);
    return x;
  }
  const int first = q.t0 / kPage + 2 * s;   // above u only if tok_off does not rise from 0
  if (u < first || (s == 0 && q.t0 > 0)) {   // rows before the first sequence's
    if (report) atomicOr(p.err, kDevErrGeometry);
    if (u < first) return x;
  }
  const int a = q.start / kPage + (u - first);     // page of the sequence
  if (q.n == 0 || a < 0 || a > (q.start + q.n - 1) / kPage) return x;
  const int page = __ldg(p.seqs.page_ids + q.p0 + a);
  if (page < 0 || page >= p.num_pages) {
    if (report) atomicOr(p.err, kDevErrPage);
    return x;
  }
  x.page = page;
  x.s0 = max(q.start - a * kPage, 0);
  x.s1 = min(q.start + q.n - a * kPage, kPage);
  x.t0 = q.t0 + a * kPage - q.start;
  // positions outside the table are found by range, so a sum past 31 bits may not wrap back into it
  const int64_t pos = int64_t(q.pos0) + int64_t(a) * kPage;
  x.pos = int32_t(max(int64_t(-64), min(pos, int64_t(1) << 30)));
  return x;
}

// The block's scale from its new rows' largest magnitude and the scale it has.
struct Scale {
  float now, inv, ratio;
  bool regrow;           // held codes follow, times ratio
};
template <bool kIsK>
__device__ __forceinline__ Scale settle(float amax, float old, int s0, int& err) {
  const int top = kIsK ? kScaleExpMaxK : kScaleExpMaxV;
  if (amax > kE4m3Max * pow2f(top)) err |= kDevErrRange;
  const float need = pow2f(scale_exp(amax, top));
  if (s0 == 0) old = 0.f;
  if (!(old >= 0.f && old < INFINITY)) { old = need; err |= kDevErrRange; }   // not a scale: the held codes stay
  Scale s;
  s.now = fmaxf(old, need);
  s.inv = __frcp_rn(s.now);   // exact for the powers of two that this kernel writes
  s.regrow = s0 > 0 && s.now != old;
  s.ratio = s.regrow ? __fdiv_rn(old, s.now) : 1.f;
  return s;
}
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float ratio) {
  const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2(w & 0xffffu)), b = f16x2_to_f32x2(e4m3x2_to_f16x2(w >> 16));
  return e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// Row `slot` of a K block turned by its position (outside the table: zeros).
__device__ __forceinline__ void turned(const AppendParams& p, const Unit& u, const float4* tab, int slot, int c,
                                       const Raw& r, float2* x, int& err) {
  Vec<__nv_bfloat16>::unpack(r.a, x);
  Vec<__nv_bfloat16>::unpack(r.b, x + 4);
  if (!p.rope) return;
  if (u.pos + slot < 0 || u.pos + slot >= p.n_pos) {
    err |= kDevErrGeometry;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = make_float2(0.f, 0.f);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) turn2(x[j], x[4 + j], tab[slot * 32 + j * 8 + c]);
  }
}

// inf saturates; nan is stored as 0 (a nan code in V would reach, as 0 * nan,
// rows whose mask hides it).
__device__ __forceinline__ void no_nan(float2* x) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (x[j].x != x[j].x) x[j].x = 0.f;
    if (x[j].y != x[j].y) x[j].y = 0.f;
  }
}

template <bool kIsK>
__device__ __forceinline__ void store_block(const AppendParams& p, const Unit& u, const float4* tab, int h, int lane,
                                            int& err) {
  const int c = lane & 7, sub = lane >> 3;
  const int H = p.num_kv_heads;
  const uint8_t* src = (kIsK ? p.k : p.v) + int64_t(h) * (kHeadDim * 2) + 16 * c;
  const int64_t stride = kIsK ? p.k_stride : p.v_stride;
  const int64_t block = (int64_t(p.layer) * p.num_pages + u.page) * H + h;
  uint8_t* codes = (kIsK ? p.pool_k : p.pool_v) + block * (kPage * kHeadDim) + 8 * c;
  float* scale_at = (kIsK ? p.k_scale : p.v_scale) + block;
  float old = u.s0 > 0 ? *scale_at : 0.f;

  Raw raw[4];
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int slot = 4 * it + sub;
    if (slot >= u.s0 && slot < u.s1) raw[it] = load_raw(src + int64_t(u.t0 + slot) * stride, kHeadDim);
  }
  float amax = 0.f;
  bool odd = false;   // a value is not finite
  if (kIsK) {
    float amin = 0.f;
    const float2 zero = make_float2(0.f, 0.f);
    float2 sum = zero;                          // of x * 0: nan when an x is not finite
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int slot = 4 * it + sub;
      if (slot >= u.s0 && slot < u.s1) {
        float2 x[8];
        turned(p, u, tab, slot, c, raw[it], x, err);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum = ffma2(x[j], zero, sum);
          amax = fmax3(amax, x[j].x, x[j].y);
          amin = fmin3(amin, x[j].x, x[j].y);
        }
      }
    }
    amax = fmaxf(amax, -amin);
    odd = !(sum.x + sum.y == 0.f);
  } else {
    uint32_t big = 0;                           // the largest magnitudes' bits, as bf16 pairs
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int slot = 4 * it + sub;
      if (slot >= u.s0 && slot < u.s1) {
        if (p.rope && (u.pos + slot < 0 || u.pos + slot >= p.n_pos)) {
          err |= kDevErrGeometry;
          raw[it] = Raw{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        }
        const uint32_t w[8] = {raw[it].a.x, raw[it].a.y, raw[it].a.z, raw[it].a.w,
                               raw[it].b.x, raw[it].b.y, raw[it].b.z, raw[it].b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) big = __vmaxu2(big, w[j] & 0x7fff7fffu);
      }
    }
    const uint32_t top = max(big >> 16, big & 0xffffu);
    odd = top >= 0x7f80u;
    amax = __uint_as_float(top << 16);
  }
  if (__any_sync(0xffffffffu, odd)) {           // rare: the scale follows the finite values
    if (odd) err |= kDevErrRange;
    amax = 0.f;
#pragma unroll 1
    for (int it = 0; it < 4; ++it) {
      const int slot = 4 * it + sub;
      if (slot >= u.s0 && slot < u.s1) {
        const Raw r = it == 0 ? raw[0] : it == 1 ? raw[1] : it == 2 ? raw[2] : raw[3];
        float2 x[8];
        Vec<__nv_bfloat16>::unpack(r.a, x);
        Vec<__nv_bfloat16>::unpack(r.b, x + 4);
        if (kIsK) turned(p, u, tab, slot, c, r, x, err);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (fabsf(x[j].x) < INFINITY) amax = fmaxf(amax, fabsf(x[j].x));
          if (fabsf(x[j].y) < INFINITY) amax = fmaxf(amax, fabsf(x[j].y));
        }
      }
    }
  }
  const bool any_odd = __any_sync(0xffffffffu, odd);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const Scale sc = settle<kIsK>(amax, old, u.s0, err);
  const float2 inv2 = make_float2(sc.inv, sc.inv);
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int slot = 4 * it + sub;
    uint2* at0 = reinterpret_cast<uint2*>(codes + slot * kHeadDim);
    uint2* at1 = reinterpret_cast<uint2*>(codes + slot * kHeadDim + 64);
    if (slot >= u.s0 && slot < u.s1) {
      float2 x[8];
      if (kIsK) {
        turned(p, u, tab, slot, c, raw[it], x, err);
      } else {
        Vec<__nv_bfloat16>::unpack(raw[it].a, x);
        Vec<__nv_bfloat16>::unpack(raw[it].b, x + 4);
      }
      if (any_odd) no_nan(x);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y0 = fmul2(x[2 * j], inv2), y1 = fmul2(x[2 * j + 1], inv2);
        w[j] = e4m3x4(y0.x, y0.y, y1.x, y1.y);
      }
      *at0 = make_uint2(w[0], w[1]);
      *at1 = make_uint2(w[2], w[3]);
    } else if (slot < u.s0) {
      if (sc.regrow) {
        uint2 w[2] = {*at0, *at1};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          w[k].x = rescaled(w[k].x, sc.ratio);
          w[k].y = rescaled(w[k].y, sc.ratio);
        }
        *at0 = w[0];
        *at1 = w[1];
      }
    } else if (u.s0 == 0) {
      *at0 = make_uint2(0u, 0u);
      *at1 = make_uint2(0u, 0u);
    }
  }
  if (lane == 0 && (u.s0 == 0 || sc.regrow)) *scale_at = sc.now;
}

}  // namespace

// heads_split blocks share a group of units: block y takes page blocks 8 y ..
// 8 y + 7, 8 (y + heads_split) .. of each, a warp a block.
__global__ void __launch_bounds__(kAppendThreads, 2) kv8_append_kernel(const AppendParams p) {
  __shared__ Tok toks[kMaxTokensPerBlock];
  __shared__ Unit units[kMaxTokensPerBlock];
  __shared__ float4 tab[2 * kPage * 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (int(blockIdx.x) >= p.kv_blocks) {
    store_rows<__nv_bfloat16, kHeadDim, false>(p, toks, tab, (int(blockIdx.x) - p.kv_blocks) * p.tokens_per_block,
                                     p.tokens_per_block);
    return;
  }
  const int u0 = int(blockIdx.x) / p.heads_split * p.units_per_block;
  const int y = int(blockIdx.x) % p.heads_split;
  if (warp < p.units_per_block) {
    const Unit u = unit_of(p, u0 + warp, lane);
    if (lane == 0) units[warp] = u;
  }
  __syncthreads();
  int err = 0;
  const int H = p.num_kv_heads;
  // The table buffers alternate with the units that have work: between two fills
  // of one buffer lies the barrier of the unit between them, which every warp
  // reaches only when it has read the first. (By the unit's number they would
  // not: a unit without a page has no barrier.)
  float4* rows = tab;
  for (int i = 0; i < p.units_per_block; ++i) {
    const Unit u = units[i];
    if (u.page < 0) continue;
    rows = rows == tab ? tab + kPage * 32 : tab;
    if (p.rope) {
      for (int f = u.s0 * 32 + tid; f < u.s1 * 32; f += kAppendThreads) {
        const int pos = u.pos + (f >> 5);
        if (pos >= 0 && pos < p.n_pos)
          rows[(f & ~31) + tab_at<8>(f & 31, 8)] =
              tab_vec(reinterpret_cast<const float4*>(p.rope + int64_t(pos) * (kHeadDim / 2)) + (f & 31));
      }
    }
    __syncthreads();
    for (int r = 8 * y + warp; r < 2 * H; r += 8 * p.heads_split) {
      if (r < H) store_block<true>(p, u, rows, r, lane, err);
      else store_block<false>(p, u, rows, r - H, lane, err);
    }
  }
  if (err && p.err) atomicOr(p.err, err);
}

// Many tokens: the same work with the rows streamed through shared memory. A
// stage is the 16 slots of 8 page blocks (K heads, then V heads of a unit):
// one bulk copy per slot and tensor brings a token's neighbouring heads, up to
// 2 KB, while the warps work on the stage before; two warps turn a block's rows
// from shared memory twice, for the maximum (which they exchange) and for the
// codes, so that little lives in registers and no load's latency is a warp's
// to wait for. (With the rows in registers, 65,536 tokens took 149 us: 80
// registers a lane spill, 128 leave 16 warps an SM. One warp a block: 114 us,
// 1.4 instructions a cycle from 17 warps.)
// Lane (r, c) = (lane / 16, lane % 16) of half-block b holds columns 4c.. and
// 64 + 4c.. of rows 8 b + r, 8 b + r + 2, ...
namespace {

constexpr int kStreamStages = 2;
constexpr int kStreamThreads = 16 * 32 + 32;           // two warps a page block, a producer
constexpr int kStageBytes = kPage * 8 * kHeadDim * 2;
constexpr int kStageTab = kPage * 32;                 // table rows, float4
struct StreamCtrl {
  uint64_t full[kStreamStages], empty[kStreamStages];
  Unit units[kMaxTokensPerBlock];
  float big[2][16];       // largest magnitudes of the half-blocks, by stage parity
  float big_finite[16];
  int32_t abort;
};
constexpr size_t kStreamSmem = kStreamStages * (size_t(kStageBytes) + kStageTab * sizeof(float4)) + sizeof(StreamCtrl) + 64;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Four values of each half of a row: x[0], x[1] | x[2], x[3].
__device__ __forceinline__ void row_words(const uint8_t* at, uint32_t* u) {
  const uint2 a = *reinterpret_cast<const uint2*>(at), b = *reinterpret_cast<const uint2*>(at + kHeadDim);
  u[0] = a.x; u[1] = a.y; u[2] = b.x; u[3] = b.y;
}

// kPlain: all 16 slots are new and their positions lie inside the table. False:
// the block's other warp gave up a wait.
template <bool kIsK, bool kPlain>
__device__ __forceinline__ bool stream_block(const AppendParams& p, const Unit& u, const uint8_t* rows,
                                             const float4* tab, int h, int warp, int lane, float* big,
                                             float* big_finite, int& err) {
  bool told = false;
  const int c = lane & 15, sub = (warp & 1) * 8 + (lane >> 4);   // first row
  constexpr int kIts = 4;                                        // rows sub, sub + 2, sub + 4, sub + 6
  const int64_t block = (int64_t(p.layer) * p.num_pages + u.page) * p.num_kv_heads + h;
  uint8_t* codes = (kIsK ? p.pool_k : p.pool_v) + block * (kPage * kHeadDim) + sub * kHeadDim + 4 * c;
  float* scale_at = (kIsK ? p.k_scale : p.v_scale) + block;
  const float old = !kPlain && u.s0 > 0 ? *scale_at : 0.f;
  rows += sub * (8 * kHeadDim * 2) + 8 * c;
  tab += sub * 32 + c;
  const bool turning = kIsK && p.rope != nullptr;
  auto is_new = [&](int i) { return kPlain || (2 * i + sub >= u.s0 && 2 * i + sub < u.s1); };
  auto outside = [&](int i) {
    return !kPlain && p.rope && (u.pos + 2 * i + sub < 0 || u.pos + 2 * i + sub >= p.n_pos);
  };
  // values of row 2 i + sub, turned; outside the table: zeros
  auto values = [&](int i, float2* x) {
    uint32_t w[4];
    row_words(rows + i * (2 * 8 * kHeadDim * 2), w);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    if (outside(i)) {
      err |= kDevErrGeometry;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = make_float2(0.f, 0.f);
    } else if (turning) {
      turn2(x[0], x[2], tab[i * 64]);
      turn2(x[1], x[3], tab[i * 64 + 16]);
    }
  };
  float amax = 0.f;
  bool odd;   // a value is not finite
  if (kIsK) {
    float amin = 0.f;
#pragma unroll(kPlain ? kIts : 1)
    for (int i = 0; i < kIts; ++i) {
      if (!is_new(i)) continue;
      float2 x[4];
      values(i, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        amax = fmax3_nan(amax, x[j].x, x[j].y);
        amin = fmin3(amin, x[j].x, x[j].y);
      }
    }
    amax = fmax3_nan(amax, -amin, 0.f);
    odd = !(amax < INFINITY);
  } else {
    uint32_t big = 0;                           // the largest magnitudes' bits, as bf16 pairs
#pragma unroll(kPlain ? kIts : 1)
    for (int i = 0; i < kIts; ++i) {
      if (!is_new(i) || outside(i)) continue;
      uint32_t w[4];
      row_words(rows + i * (2 * 8 * kHeadDim * 2), w);
#pragma unroll
      for (int j = 0; j < 4; ++j) big = __vmaxu2(big, w[j] & 0x7fff7fffu);
    }
    const uint32_t top = max(big >> 16, big & 0xffffu);
    odd = top >= 0x7f80u;
    amax = __uint_as_float(top << 16);
  }
  // both warps' maximum; a value that is not finite makes it infinite
  auto shared_max = [&](float m, float* at) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) at[warp] = m;
    told = named_bar_leave(1 + (warp >> 1), 64, false);
    return fmaxf(at[warp & ~1], at[warp | 1]);
  };
  if (odd) err |= kDevErrRange;
  amax = shared_max(odd ? INFINITY : amax, big);
  if (told) return false;                       // no wait lies between this round and the block's others
  const bool any_odd = amax == INFINITY;
  if (any_odd) {                                // rare: the scale follows the finite values
    amax = 0.f;
#pragma unroll 1
    for (int i = 0; i < kIts; ++i) {
      if (!is_new(i)) continue;
      float2 x[4];
      values(i, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (fabsf(x[j].x) < INFINITY) amax = fmaxf(amax, fabsf(x[j].x));
        if (fabsf(x[j].y) < INFINITY) amax = fmaxf(amax, fabsf(x[j].y));
      }
    }
    amax = shared_max(amax, big_finite);
    named_bar_sync(1 + (warp >> 1), 64);        // both have read it before the next block's turn
  }
  const Scale sc = settle<kIsK>(amax, old, kPlain ? 0 : u.s0, err);
  const float2 inv2 = make_float2(sc.inv, sc.inv);
#pragma unroll(kPlain ? kIts : 1)
  for (int i = 0; i < kIts; ++i) {
    uint32_t* at0 = reinterpret_cast<uint32_t*>(codes + 2 * i * kHeadDim);
    uint32_t* at1 = at0 + 16;
    if (is_new(i)) {
      float2 x[4];
      values(i, x);
      if (any_odd) {   // inf saturates, nan becomes 0
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (x[j].x != x[j].x) x[j].x = 0.f;
          if (x[j].y != x[j].y) x[j].y = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = fmul2(x[j], inv2);
      *at0 = e4m3x4(x[0].x, x[0].y, x[1].x, x[1].y);
      *at1 = e4m3x4(x[2].x, x[2].y, x[3].x, x[3].y);
    } else if (2 * i + sub < u.s0) {
      if (sc.regrow) {
        *at0 = rescaled(*at0, sc.ratio);
        *at1 = rescaled(*at1, sc.ratio);
      }
    } else if (u.s0 == 0) {
      *at0 = 0u;
      *at1 = 0u;
    }
  }
  if (lane == 0 && !(warp & 1) && (kPlain || u.s0 == 0 || sc.regrow)) *scale_at = sc.now;
  return true;
}

}  // namespace

__global__ void __launch_bounds__(kStreamThreads, 2) kv8_append_stream_kernel(const AppendParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((16 - (smem_u32(smem_raw) & 15)) & 15);
  float4* tabs = reinterpret_cast<float4*>(smem + kStreamStages * kStageBytes);
  StreamCtrl* ctl = reinterpret_cast<StreamCtrl*>(tabs + kStreamStages * kStageTab);
  if (p.q) pdl_launch_dependents();   // the queries' kernel, which waits for this one at its end
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kStreamStages; ++s) {
      mbar_init(&ctl->full[s], 2);     // the copies' bytes and the table rows
      mbar_init(&ctl->empty[s], 16);
    }
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp < p.units_per_block) {
    const Unit u = unit_of(p, int(blockIdx.x) / p.heads_split * p.units_per_block + warp, lane);
    if (lane == 0) ctl->units[warp] = u;
  }
  __syncthreads();
  volatile int* abort_flag = &ctl->abort;
  const int H = p.num_kv_heads;
  const int groups = (2 * H + 7) / 8;   // stages of a unit, shared by heads_split blocks
  const int y0 = int(blockIdx.x) % p.heads_split;
  if (warp == 16) {
    uint32_t n = 0;
    bool bad = false;
    for (int i = 0; i < p.units_per_block && !bad; ++i) {
      const Unit u = ctl->units[i];
      if (u.page < 0) continue;
      for (int y = y0; y < groups; y += p.heads_split, ++n) {
        const int s = n % kStreamStages;
        if (n >= uint32_t(kStreamStages) && !mbar_wait(&ctl->empty[s], (n / kStreamStages - 1) & 1, abort_flag)) {
          bad = true;
          break;
        }
        __syncwarp();
        const int r0 = 8 * y, r1 = min(r0 + 8, 2 * H);
        const int nk = max(min(r1, H) - r0, 0), nv = r1 - r0 - nk;    // K heads, then V heads
        if (lane == 0) mbar_arrive_expect_tx(&ctl->full[s], uint32_t((u.s1 - u.s0) * (r1 - r0) * kHeadDim * 2));
        __syncwarp();
        if (lane >= u.s0 && lane < u.s1) {
          uint8_t* dst = smem + s * kStageBytes + lane * (8 * kHeadDim * 2);
          const int64_t t = u.t0 + lane;
          if (nk > 0) bulk_load(dst, p.k + t * p.k_stride + int64_t(r0) * kHeadDim * 2, nk * kHeadDim * 2, &ctl->full[s]);
          if (nv > 0)
            bulk_load(dst + nk * kHeadDim * 2, p.v + t * p.v_stride + int64_t(r0 + nk - H) * kHeadDim * 2,
                      nv * kHeadDim * 2, &ctl->full[s]);
        }
        if (p.rope && nk > 0) {
          float4* rows = tabs + s * kStageTab;
#pragma unroll 8
          for (int slot = u.s0; slot < u.s1; ++slot) {
            const int pos = u.pos + slot;
            if (pos >= 0 && pos < p.n_pos)
              rows[slot * 32 + tab_at<4>(lane, 16)] =
                  tab_vec(reinterpret_cast<const float4*>(p.rope + int64_t(pos) * (kHeadDim / 2)) + lane);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->full[s]);
      }
    }
    if (bad) {
      if (lane == 0 && p.err) atomicOr(p.err, kDevErrTimeout);
      ctl->abort = 1;
    }
    // Let every copy this warp issued land before the block exits, whether a
    // warp has given up by now or does so later. (They have landed, or the others
    // still wait for them: it costs nothing.)
    if (lane == 0) {
      int zero = 0;
      for (uint32_t t = n > kStreamStages ? n - kStreamStages : 0; t < n; ++t)
        mbar_wait(&ctl->full[t % kStreamStages], (t / kStreamStages) & 1, &zero);
    }
    __syncwarp();
    return;
  }
  uint32_t n = 0;
  int err = 0;
  Run run = Run::kOn;   // the two warps of a page block share a named barrier
  for (int i = 0; i < p.units_per_block && run == Run::kOn; ++i) {
    const Unit u = ctl->units[i];
    if (u.page < 0) continue;
    for (int y = y0; y < groups; y += p.heads_split, ++n) {
      const int s = n % kStreamStages;
      if (!mbar_wait(&ctl->full[s], (n / kStreamStages) & 1, abort_flag)) {
        ctl->abort = 1;
        err |= kDevErrTimeout;
        run = Run::kGaveUp;
        break;
      }
      const int r = 8 * y + (warp >> 1);
      const uint8_t* rows = smem + s * kStageBytes + (warp >> 1) * (kHeadDim * 2);
      const float4* tab = tabs + s * kStageTab;
      float* big = ctl->big[n & 1];
      const bool plain = u.s0 == 0 && u.s1 == kPage && (!p.rope || (u.pos >= 0 && u.pos + kPage <= p.n_pos));
      bool on = true;
      if (r < H) {
        on = plain ? stream_block<true, true>(p, u, rows, tab, r, warp, lane, big, ctl->big_finite, err)
                   : stream_block<true, false>(p, u, rows, tab, r, warp, lane, big, ctl->big_finite, err);
      } else if (r < 2 * H) {
        on = plain ? stream_block<false, true>(p, u, rows, tab, r - H, warp, lane, big, ctl->big_finite, err)
                   : stream_block<false, false>(p, u, rows, tab, r - H, warp, lane, big, ctl->big_finite, err);
      }
      if (!on) {
        run = Run::kTold;
        break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->empty[s]);
    }
  }
  if (run != Run::kTold) named_bar_leave(1 + (warp >> 1), 64, run == Run::kGaveUp);
  if (err && p.err) atomicOr(p.err, err);
}

// Queries alone, beside the streamed cache blocks of a call with many tokens:
// the stream kernel releases this one as soon as its blocks have started, and
// this one completes only after it, so that whatever follows finds both done.
__global__ void __launch_bounds__(kAppendThreads, 4) rope_q_kernel(const AppendParams p) {
  __shared__ Tok toks[kMaxTokensPerBlock];
  __shared__ float4 tab[kMaxTokensPerBlock * 32];
  store_rows<__nv_bfloat16, kHeadDim, false>(p, toks, tab, int(blockIdx.x) * p.tokens_per_block, p.tokens_per_block);
  pdl_wait();
}

// (cos, sin) of position p and pair i: the angle p * base^(-2 i / d), in fp64,
// each stored as the nearest fp32 value.
__global__ void __launch_bounds__(256) rope_cos_sin_kernel(double base, int half, int64_t n, float2* table) {
  const int64_t x = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (x >= n) return;
  const double theta = pow(base, -double(x % half) / double(half));
  double sn, cn;
  sincos(double(x / half) * theta, &sn, &cn);
  table[x] = make_float2(float(cn), float(sn));
}

// The kernels below write pool pages and queries that the next kernel may read
// before its own wait, so they release no dependents early (the stream kernel
// only the queries' kernel of its own call) and start only once the kernel
// before them has completed.
cudaError_t launch_kv_append(const AppendParams& p, int is_f32, int grid, cudaStream_t stream) {
  const auto kernel = !is_f32               ? kv_append_kernel<__nv_bfloat16, 128>
                      : p.head_dim == 128 ? kv_append_kernel<float, 128>
                                          : kv_append_kernel<float, 64>;
  return launch_plain(kernel, dim3(grid), dim3(kAppendThreads), 0, stream, p);
}
cudaError_t launch_kv8_append(const AppendParams& p, int grid, cudaStream_t stream) {
  return launch_plain(kv8_append_kernel, dim3(grid), dim3(kAppendThreads), 0, stream, p);
}
cudaError_t launch_kv8_append_stream(const AppendParams& p, int grid, cudaStream_t stream) {
  static SmemAttr attr;
  const cudaError_t e = ensure_smem_attr(kv8_append_stream_kernel, attr, kStreamSmem);
  if (e != cudaSuccess) return e;
  return launch_plain(kv8_append_stream_kernel, dim3(grid), dim3(kStreamThreads), kStreamSmem, stream, p);
}
cudaError_t launch_rope_q(const AppendParams& p, int grid, cudaStream_t stream) {
  return launch_pdl(rope_q_kernel, dim3(grid), dim3(kAppendThreads), 0, stream, 1, p);
}
cudaError_t launch_rope_cos_sin(double base, int head_dim, int n_pos, float2* table, cudaStream_t stream) {
  const int64_t n = int64_t(n_pos) * (head_dim / 2);
  return launch_plain(rope_cos_sin_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, stream, base, head_dim / 2, n,
                      table);
}

}  // namespace rag
