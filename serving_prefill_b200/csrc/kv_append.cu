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
#include "params.cuh"

namespace rag {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxTokensPerBlock = 8;

struct Tok {
  int64_t page;      // -1: not stored
  int32_t slot;
  int32_t pos;       // row of the table; -1: outside it (the row becomes zeros)
  int32_t tail;      // slots behind this token to zero
  int32_t live;      // 0: a row behind the last sequence
};

// Last s with tok_off[s] <= t (0 when there is none).
__device__ __forceinline__ int seq_of(const AppendSeqs& a, int t) {
  int lo = 0, hi = a.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.tok_off + mid) <= t) lo = mid; else hi = mid - 1;
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
  q.ok = q.t0 >= 0 && q.n >= 0 && t1 <= a.total_new && q.start >= 0 && q.p0 >= 0 && q.n_pages >= 0 &&
         p1 <= a.total_pages && int64_t(q.start) + q.n <= int64_t(q.n_pages) * kPage;
  return q;
}

__device__ __forceinline__ Tok token_of(const AppendParams& p, int t, bool report) {
  Tok k;
  k.page = -1; k.slot = 0; k.pos = -1; k.tail = 0; k.live = 0;
  if (t >= p.seqs.total_new || t >= __ldg(p.seqs.tok_off + p.seqs.n_seqs)) return k;
  k.live = 1;
  const Seq q = load_seq(p.seqs, seq_of(p.seqs, t));
  const int at = t - q.t0;
  if (!q.ok || at < 0 || at >= q.n) {
    if (report && p.err) atomicOr(p.err, kDevErrGeometry);
    return k;
  }
  const int i = q.start + at;
  const int64_t pos = int64_t(q.pos0) + i;
  if (!p.rope) {
    k.pos = 0;
  } else if (pos >= 0 && pos < p.n_pos) {
    k.pos = int32_t(pos);
  } else if (report && p.err) {
    atomicOr(p.err, kDevErrGeometry);
  }
  const int page = __ldg(p.seqs.page_ids + q.p0 + i / kPage);
  if (page < 0 || page >= p.num_pages) {
    if (report && p.err) atomicOr(p.err, kDevErrPage);
    return k;
  }
  k.page = page;
  k.slot = i % kPage;
  const bool last = at == q.n - 1;
  if (last && i - k.slot >= q.start) k.tail = kPage - 1 - k.slot;
  return k;
}

// The two products' rounding is part of the operator (see above).
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float na = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  const float nb = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
  a = na;
  b = nb;
}

// 16 bytes of a row's first half and of its second half as fp32 pairs.
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void load(const uint8_t* at, float* x) {
    const uint4 w = *reinterpret_cast<const uint4*>(at);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(u[j] << 16);
      x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(uint8_t* at, const float* x) {
    *reinterpret_cast<uint4*>(at) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                               pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
};
template <> struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void load(const uint8_t* at, float* x) {
    const float4 w = *reinterpret_cast<const float4*>(at);
    x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
  }
  static __device__ __forceinline__ void store(uint8_t* at, const float* x) {
    *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
// V of a bf16 cache is stored as fp16 (saturated, reported).
__device__ __forceinline__ void store_f16(uint8_t* at, const float* x, bool& over) {
#pragma unroll
  for (int j = 0; j < 8; ++j) over = over || !(fabsf(x[j]) < 65520.f);
  *reinterpret_cast<uint4*>(at) = make_uint4(pack_f16x2_sat(x[0], x[1]), pack_f16x2_sat(x[2], x[3]),
                                             pack_f16x2_sat(x[4], x[5]), pack_f16x2_sat(x[6], x[7]));
}

template <typename T>
__device__ __forceinline__ void rotate_row(const AppendParams& p, int pos, int c, float* a, float* b) {
  constexpr int N = Vec<T>::kN;
  if (pos < 0) {
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] = b[j] = 0.f;
  } else if (p.rope) {
    const float4* cs = reinterpret_cast<const float4*>(p.rope + int64_t(pos) * (p.head_dim / 2) + c * N);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float4 w = __ldg(cs + j);
      turn(a[2 * j], b[2 * j], make_float2(w.x, w.y));
      turn(a[2 * j + 1], b[2 * j + 1], make_float2(w.z, w.w));
    }
  }
}

// Row `h` of token t of q, rotated to q_out (dense [total_new][H_q][d]).
template <typename T>
__device__ __forceinline__ void q_row(const AppendParams& p, const Tok& k, int t, int h, int c) {
  constexpr int N = Vec<T>::kN;
  const int half = p.head_dim / 2;
  float a[N], b[N];
  const uint8_t* src = p.q + int64_t(t) * p.q_stride + (int64_t(h) * p.head_dim + c * N) * sizeof(T);
  Vec<T>::load(src, a);
  Vec<T>::load(src + half * sizeof(T), b);
  rotate_row<T>(p, k.pos, c, a, b);
  uint8_t* dst = p.q_out + ((int64_t(t) * p.num_q_heads + h) * p.head_dim + c * N) * sizeof(T);
  Vec<T>::store(dst, a);
  Vec<T>::store(dst + half * sizeof(T), b);
}

}  // namespace

// A block stores tokens_per_block tokens: their descriptors are resolved once
// into shared memory, then groups of d/2 / (16 / sizeof(T)) lanes take a row
// (K heads, V heads, query heads of each token in turn).
template <typename T>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
  constexpr int N = Vec<T>::kN;
  __shared__ Tok toks[kMaxTokensPerBlock];
  const int t0 = blockIdx.x * p.tokens_per_block;
  if (threadIdx.x < p.tokens_per_block) toks[threadIdx.x] = token_of(p, t0 + threadIdx.x, true);
  __syncthreads();
  const int half = p.head_dim / 2;
  const int lanes = half / N;                      // lanes of one row
  const int c = threadIdx.x % lanes;
  const int groups = kAppendThreads / lanes;
  const int H = p.num_kv_heads;
  const int rows = 2 * H + (p.q ? p.num_q_heads : 0);
  const int64_t row_bytes = int64_t(p.head_dim) * sizeof(T);
  bool over = false;
  for (int x = threadIdx.x / lanes; x < rows * p.tokens_per_block; x += groups) {
    const int n = x / rows, r = x % rows;
    const Tok k = toks[n];
    const int t = t0 + n;
    if (!k.live) continue;
    if (r >= 2 * H) {
      q_row<T>(p, k, t, r - 2 * H, c);
      continue;
    }
    if (k.page < 0) continue;
    const bool is_k = r < H;
    const int h = is_k ? r : r - H;
    float a[N], b[N];
    const uint8_t* src = (is_k ? p.k + int64_t(t) * p.k_stride : p.v + int64_t(t) * p.v_stride) + h * row_bytes +
                         c * N * int(sizeof(T));
    Vec<T>::load(src, a);
    Vec<T>::load(src + half * sizeof(T), b);
    if (is_k || k.pos < 0) rotate_row<T>(p, k.pos, c, a, b);
    uint8_t* dst = (is_k ? p.pool_k : p.pool_v) +
                   (((int64_t(p.layer) * p.num_pages + k.page) * H + h) * kPage + k.slot) * row_bytes +
                   c * N * int(sizeof(T));
    if (sizeof(T) == 2 && !is_k) {
      store_f16(dst, a, over);
      store_f16(dst + half * sizeof(T), b, over);
    } else {
      Vec<T>::store(dst, a);
      Vec<T>::store(dst + half * sizeof(T), b);
    }
  }
  // slots behind a sequence's last token in a page this call began
  for (int n = 0; n < p.tokens_per_block; ++n) {
    const Tok k = toks[n];
    if (k.page < 0 || k.tail == 0) continue;
    const int vecs = int(k.tail * row_bytes / 16);
    for (int x = threadIdx.x; x < 2 * H * vecs; x += kAppendThreads) {
      const int h = x / vecs % H;
      uint8_t* base = (x / vecs < H ? p.pool_k : p.pool_v) +
                      (((int64_t(p.layer) * p.num_pages + k.page) * H + h) * kPage + k.slot + 1) * row_bytes;
      reinterpret_cast<uint4*>(base)[x % vecs] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (over && p.err) atomicOr(p.err, kDevErrRange);
}

// 8-bit pool. A warp owns one (page the call touches, KV head) of K or of V:
// the block scale needs the largest magnitude of all its new rows, and a scale
// that grows has to bring the page's held codes along, so the page block is
// the unit that one warp can settle alone, with no atomics and no second pass.
// The unit's pages are found without a prefix kernel: sequence s owns the unit
// numbers from tok_off[s] / 16 + 2 s on, which leaves room for every page that
// its n tokens can touch ((n + 14) / 16 + 1 at most); units past a sequence's
// last page have nothing to do. Lane (r, c) = (lane / 8, lane % 8) holds
// columns 8c.. and 64 + 8c.. of rows r, r + 4, r + 8, r + 12.
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane & 7, sub = lane >> 3;
  const int H = p.num_kv_heads;
  if (int(blockIdx.x) >= p.kv_blocks) {
    // the queries: a group of 8 lanes per row
    __shared__ Tok toks[kMaxTokensPerBlock];
    const int t0 = (int(blockIdx.x) - p.kv_blocks) * p.tokens_per_block;
    if (threadIdx.x < p.tokens_per_block) toks[threadIdx.x] = token_of(p, t0 + threadIdx.x, false);
    __syncthreads();
    for (int x = threadIdx.x >> 3; x < p.num_q_heads * p.tokens_per_block; x += kAppendThreads / 8) {
      const int n = x / p.num_q_heads;
      if (toks[n].live) q_row<__nv_bfloat16>(p, toks[n], t0 + n, x % p.num_q_heads, c);
    }
    return;
  }
  const int64_t task = int64_t(blockIdx.x) * (kAppendThreads / 32) + warp;
  const int u = int(task / (2 * H));
  const int r = int(task % (2 * H));
  const bool is_k = r < H;
  const int h = is_k ? r : r - H;
  // last sequence whose first unit is at or before u
  int lo = 0, hi = p.seqs.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.seqs.tok_off + mid) / kPage + 2 * mid <= u) lo = mid; else hi = mid - 1;
  }
  const Seq q = load_seq(p.seqs, lo);
  if (!q.ok) {
    if (lane == 0 && p.err) atomicOr(p.err, kDevErrGeometry);
    return;
  }
  const int a = q.start / kPage + (u - (q.t0 / kPage + 2 * lo));     // page of the sequence
  if (q.n == 0 || a < 0 || a > (q.start + q.n - 1) / kPage) return;
  const int s0 = max(q.start - a * kPage, 0);                         // slots [s0, s1) are new
  const int s1 = min(q.start + q.n - a * kPage, kPage);
  const int page = __ldg(p.seqs.page_ids + q.p0 + a);
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0 && p.err) atomicOr(p.err, kDevErrPage);
    return;
  }
  const int64_t block = (int64_t(p.layer) * p.num_pages + page) * H + h;
  uint8_t* codes = (is_k ? p.pool_k : p.pool_v) + block * (kPage * kHeadDim);
  float* scale_at = (is_k ? p.k_scale : p.v_scale) + block;
  float old = s0 > 0 ? *scale_at : 0.f;

  float x[4][16];
  float amax = 0.f;
  int err = 0;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int slot = 4 * it + sub;
    const bool have = slot >= s0 && slot < s1;
    if (have) {
      const int i = a * kPage + slot;                                 // token of the sequence
      const int t = q.t0 + i - q.start;
      const uint8_t* src = (is_k ? p.k + int64_t(t) * p.k_stride : p.v + int64_t(t) * p.v_stride) +
                           (int64_t(h) * kHeadDim + 8 * c) * 2;
      Vec<__nv_bfloat16>::load(src, x[it]);
      Vec<__nv_bfloat16>::load(src + kHeadDim, x[it] + 8);
      const int64_t pos = int64_t(q.pos0) + i;
      const bool inside = !p.rope || (pos >= 0 && pos < p.n_pos);
      if (!inside) err |= kDevErrGeometry;
      if (is_k || !inside) rotate_row<__nv_bfloat16>(p, inside ? (p.rope ? int(pos) : 0) : -1, c, x[it], x[it] + 8);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float m = fabsf(x[it][j]);
        if (m < INFINITY) {
          amax = fmaxf(amax, m);
        } else {
          // inf saturates; nan is stored as 0 (a nan code in V would reach,
          // as 0 * nan, rows whose mask hides it). Both are reported.
          err |= kDevErrRange;
          if (m != m) x[it][j] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int top = is_k ? kScaleExpMaxK : kScaleExpMaxV;
  if (amax > kE4m3Max * pow2f(top)) err |= kDevErrRange;
  const float need = pow2f(scale_exp(amax, top));
  if (!(old >= 0.f && old < INFINITY)) { old = need; err |= kDevErrRange; }   // not a scale: the held codes stay
  const float now = fmaxf(old, need);
  const float inv = __frcp_rn(now);   // exact for the powers of two that this kernel writes
  const bool regrow = s0 > 0 && now != old;
  const float ratio = regrow ? __fdiv_rn(old, now) : 1.f;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int slot = 4 * it + sub;
    uint2* at0 = reinterpret_cast<uint2*>(codes + slot * kHeadDim + 8 * c);
    uint2* at1 = reinterpret_cast<uint2*>(codes + slot * kHeadDim + 64 + 8 * c);
    if (slot >= s0 && slot < s1) {
      float* y = x[it];
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] *= inv;
      *at0 = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
      *at1 = make_uint2(e4m3x4(y[8], y[9], y[10], y[11]), e4m3x4(y[12], y[13], y[14], y[15]));
    } else if (slot < s0) {
      if (regrow) {
        uint2 w[2] = {*at0, *at1};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t* v = reinterpret_cast<uint32_t*>(&w[k]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 f0 = f16x2_to_f32x2(e4m3x2_to_f16x2(v[j] & 0xffffu));
            const float2 f1 = f16x2_to_f32x2(e4m3x2_to_f16x2(v[j] >> 16));
            v[j] = e4m3x4(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio);
          }
        }
        *at0 = w[0];
        *at1 = w[1];
      }
    } else if (s0 == 0) {
      *at0 = make_uint2(0u, 0u);
      *at1 = make_uint2(0u, 0u);
    }
  }
  if (lane == 0 && (s0 == 0 || regrow)) *scale_at = now;
  if (err && p.err) atomicOr(p.err, err);
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
// before its own wait, so they release no dependents early and start only once
// the kernel before them has completed.
cudaError_t launch_kv_append(const AppendParams& p, int is_f32, int grid, cudaStream_t stream) {
  return is_f32 ? launch_plain(kv_append_kernel<float>, dim3(grid), dim3(kAppendThreads), 0, stream, p)
                : launch_plain(kv_append_kernel<__nv_bfloat16>, dim3(grid), dim3(kAppendThreads), 0, stream, p);
}
cudaError_t launch_kv8_append(const AppendParams& p, int grid, cudaStream_t stream) {
  return launch_plain(kv8_append_kernel, dim3(grid), dim3(kAppendThreads), 0, stream, p);
}
cudaError_t launch_rope_cos_sin(double base, int head_dim, int n_pos, float2* table, cudaStream_t stream) {
  const int64_t n = int64_t(n_pos) * (head_dim / 2);
  return launch_plain(rope_cos_sin_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, stream, base, head_dim / 2, n,
                      table);
}

}  // namespace rag
