// Attention over the 8-bit pool for short query blocks: at most 16 rows (query
// tokens x the query heads of one KV head) per unit, as in a generation step
// (the softmax(Q K^T / sqrt(d_k) + M) V of kv8_fwd.cu).
//
// The products are transposed so that a thread owns a key, and neither K nor V
// is ever converted: both tiles go from TMA to the tensor core as codes.
//   S^T = K8 [Q_hi; Q_lo]^T   A = the K tile, B = the rows' two e4m3 parts (lo
//         times 16), each part in columns of its own
//   p = 2^(score + log2(scale of V's page) - m + 6) per key and row: the V scale
//         is folded into the weight, so that pages of any scale share one
//         accumulator; the row sum takes p / scale
//   p = hi + mid / 16 + lo / 256, three e4m3 parts (at least 11 bits; the least
//         part that counts is 2^-24 of the row's largest weight), P^T rows of
//         their own in shared memory
//   O^T += V8^T [P_hi; P_mid; P_lo]^T   A = the V tile read as [d x keys]
// The parts cost only tensor-core columns, of which a step of 4 to 16 rows
// leaves the most unused; converting the tiles would cost shared-memory
// bandwidth and a warpgroup, and the kernel is there to stream HBM. Two CTAs
// share an SM, so that one's item start, tile hand-offs and epilogue run under
// the other's loads.
// Measured: 64 requests of about 12,900 keys (1.65 GB) 296 us, 0.85 of the
// measured HBM rate; 16 requests of about 3,900 keys (130 MB) 35 us, of which
// 5 to 6 us pass before the first K box is issued (loads that follow one
// another, and code that runs cold), 1.6 more until the first scores and 3 in
// the combine; one request of 560 keys 8.3 us.
// Warps: 0-3 keys, 4 producer (page table -> TMA boxes of 2 KB, scales a tile
// ahead), 5 MMA, 6 zeroes V slots that hold no token (0 * nan), 7 splits Q one
// item ahead. Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <type_traits>

#include "kv8.cuh"
#include "leave.cuh"
#include "params.cuh"

namespace rag {
namespace d8 {

constexpr int kRows = 16;                        // most rows of a unit
constexpr int kKSt = 3, kVSt = 2;                // K and V stages
constexpr int kThreads = 256;
constexpr int kQBytes = 2 * kRows * kHeadDim;    // hi and lo rows
constexpr int kPBytes = 3 * kRows * kBN;         // hi, mid and lo rows
constexpr int kDescSlots = 4;
constexpr float kRescale = 2.0f;                 // log2 units a row max may grow before O is rescaled
constexpr float kTop = 6.0f;                     // p = 2^kTop at the reference max, at most 2^(kTop + kRescale)
constexpr uint32_t kColO = 64;                   // S^T buffers at columns 0 and 32, O^T at 64 .. 111
constexpr uint32_t kTmemCols = 128;

struct TileDesc {
  float ks[kPagesPerTile];         // scale of K
  float lv[kPagesPerTile];         // log2 of the scale of V
  float iv[kPagesPerTile];         // 1 / scale of V
  int32_t lstart[kPagesPerTile];   // logical position of the page's slot 0
  uint8_t nvalid[kPagesPerTile];
};

struct Ctrl {
  uint64_t q_full[2], q_empty[2];
  uint64_t kfull[kKSt], kempty[kKSt];
  uint64_t vfull[kVSt], vempty[kVSt], vready[kVSt];
  uint64_t s_full[2], p_full[2], pv_done[2], o_full, o_free;
  uint64_t teardown;
  uint64_t desc_full[kDescSlots], desc_empty[kDescSlots];
  TileDesc desc[kDescSlots];
  ChunkCache chunks;
  Kv8Ring ring;
  alignas(8) uint8_t vnv[kVSt][kPagesPerTile];   // valid slots of a V stage's pages
  float sq[2][kRows];                 // row scale of Q times the softmax scale (log2)
  alignas(16) float red[2][kRows][4]; // per-tile row maxima of the four key warps, by tile parity
  alignas(16) float lsum[kRows][4];   // per-item row sums of the four key warps
  uint32_t tmem_base;
  int32_t abort;
};

static_assert(offsetof(Ctrl, vnv) % 8 == 0 && offsetof(Ctrl, red) % 16 == 0 && offsetof(Ctrl, lsum) % 16 == 0,
              "read as vectors");

constexpr size_t kSmemData = size_t(2) * kQBytes + 2 * kPBytes + size_t(kKSt + kVSt) * kTile8;

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// N (a multiple of 8) columns of the warp's 32 lanes
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) tmem_ld8(taddr + i, r + i);
  tmem_wait_ld();
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) tmem_st8(taddr + i, r + i);
  tmem_wait_st();
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Low words of the operands' descriptors: K, Q and P tiles are K-major rows of
// 128 codes, a k-step of 32 codes is 32 bytes on (2 in units of 16). The V tile
// [128 keys][128 d] is the MN-major A operand V^T (M = d: one 128-byte atom, no
// leading offset), a k-step of 32 keys is 4 KB on.
// Byte of (row n, column k) in a tile of 128-byte rows, 128B-swizzled.
__device__ __forceinline__ uint32_t swz(int n, int k) {
  return uint32_t((n >> 3) * 1024 + (n & 7) * 128 + (((k >> 4) ^ (n & 7)) << 4) + (k & 15));
}

// Columns of the products for rows padded to R (N is a multiple of 16).
__host__ __device__ constexpr int n_qk(int R) { return R <= 8 ? 16 : 32; }
__host__ __device__ constexpr int n_pv(int R) { return (3 * R + 15) / 16 * 16; }
__device__ __forceinline__ int pad_rows(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }

}  // namespace d8

using namespace d8;

__global__ void __launch_bounds__(d8::kThreads, 2)
kv8_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const Kv8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sK = smem;
  uint8_t* sV = sK + kKSt * kTile8;
  uint8_t* sQ = sV + kVSt * kTile8;
  uint8_t* sP = sQ + 2 * kQBytes;
  Ctrl* ctl = reinterpret_cast<Ctrl*>(sP + 2 * kPBytes);
  int32_t* prefix = reinterpret_cast<int32_t*>(ctl + 1);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int G = p.group;

  pdl_launch_dependents();

  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->q_full[b], 1);
      mbar_init(&ctl->q_empty[b], 5);   // the last QK and the four key warps (row scales)
      mbar_init(&ctl->s_full[b], 1);
      mbar_init(&ctl->p_full[b], 128);
      mbar_init(&ctl->pv_done[b], 1);
    }
    for (int s = 0; s < kKSt; ++s) { mbar_init(&ctl->kfull[s], 1); mbar_init(&ctl->kempty[s], 1); }
    for (int s = 0; s < kVSt; ++s) {
      mbar_init(&ctl->vfull[s], 1);
      mbar_init(&ctl->vempty[s], 1);
      mbar_init(&ctl->vready[s], 1);
    }
    mbar_init(&ctl->o_full, 1);
    mbar_init(&ctl->o_free, 128);
    mbar_init(&ctl->teardown, 1);
    for (int s = 0; s < kDescSlots; ++s) {
      mbar_init(&ctl->desc_full[s], 1);
      mbar_init(&ctl->desc_empty[s], 4);   // one arrival per key warp
    }
    kv8_ring_init(&ctl->ring, 7);   // 4 key warps, MMA, V and Q warps
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4 && lane == 0) { tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  volatile int* abort_flag = &ctl->abort;
  Kv8Item it = {};
  uint32_t n_it = 0;   // items taken

  if (warp < 4) {
    // ------------------------------------------------------------ key warps: thread = key of the tile
    const int k = tid;
    const uint32_t lane_off = uint32_t(warp * 32) << 16;
    uint32_t t_glob = 0, n_items = 0;
    // One item with its rows padded to R.
    auto run_item = [&](auto Rc, int n) -> Run {
      constexpr int R = decltype(Rc)::value;
      constexpr int NO = (3 * R + 7) / 8 * 8;   // O^T columns in use, to the next 8
      const int rows = it.n_q * G;
      float mm[R], ls[R];                       // reference max less kTop; row sum
#pragma unroll
      for (int r = 0; r < R; ++r) { mm[r] = -INFINITY; ls[r] = 0.f; }
      uint32_t ov[NO];
#pragma unroll
      for (int j = 0; j < NO; ++j) ov[j] = 0u;
      {
        if (!mbar_wait(&ctl->q_full[n_items & 1], (n_items >> 1) & 1, abort_flag)) return Run::kGaveUp;
        const float* sq = ctl->sq[n_items & 1];
        const int first = p.causal ? it.n_doc - it.n_q : it.n_doc;   // row r sees positions <= first + r / G
        for (int i = 0; i < n; ++i) {
          const uint32_t t = t_glob + i;
          const uint32_t slot = t % kDescSlots;
          const int bsel = int(t & 1u);
          if (!mbar_wait(&ctl->desc_full[slot], (t / kDescSlots) & 1, abort_flag)) return Run::kGaveUp;
          const TileDesc* td = &ctl->desc[slot];
          const float kf = td->ks[k >> 4], lv = td->lv[k >> 4], iv = td->iv[k >> 4];
          const int pos = td->lstart[k >> 4] + (k & 15);
          const bool kvalid = (k & 15) < int(td->nvalid[k >> 4]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->desc_empty[slot]);
          if (!mbar_wait(&ctl->s_full[bsel], (t >> 1) & 1, abort_flag)) return Run::kGaveUp;
          tc_fence_after();
          uint32_t u[2 * R];
          tmem_ldn<2 * R>(tmem + lane_off + 32u * bsel, u);
          float y[R];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bool vis = kvalid && r < rows && pos <= first + r / G;
            const float s = fmaf(__uint_as_float(u[R + r]), 0.0625f, __uint_as_float(u[r]));
            y[r] = vis ? fmaf(s, kf * sq[r], lv) : -INFINITY;
            const float mt = warp_max(y[r]);
            if (lane == 0) ctl->red[bsel][r][warp] = mt;
          }
          if (named_bar_leave(1, 128, false)) return Run::kTold;
          float alpha[R];
          bool need = false;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float4 m4 = *reinterpret_cast<const float4*>(ctl->red[bsel][r]);
            const float mt = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)) - kTop;
            alpha[r] = 1.f;
            if (mt != -INFINITY) {
              if (mm[r] == -INFINITY) {
                mm[r] = mt;   // the row's first visible key: O^T holds zeros for it so far
              } else if (mt > mm[r] + kRescale) {
                alpha[r] = ex2(mm[r] - mt);
                mm[r] = mt;
                need = true;
              }
            }
          }
          if (need) {   // the same decision in every key thread (the maxima are shared)
            // O^T must hold PV of the previous tile before it is rescaled
            if (!mbar_wait(&ctl->pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, abort_flag)) return Run::kGaveUp;
            tc_fence_after();
            tmem_ldn<NO>(tmem + lane_off + kColO, ov);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              ls[r] *= alpha[r];
#pragma unroll
              for (int j = 0; j < 3; ++j) ov[j * R + r] = __float_as_uint(__uint_as_float(ov[j * R + r]) * alpha[r]);
            }
            tmem_stn<NO>(tmem + lane_off + kColO, ov);
          }
          // this P^T buffer was last read by the PV of tile t - 2
          if (t >= 2 && !mbar_wait(&ctl->pv_done[bsel], ((t >> 1) + 1) & 1, abort_flag)) return Run::kGaveUp;
          uint8_t* pb = sP + bsel * kPBytes;
#pragma unroll
          for (int r = 0; r < R; r += 2) {
            // y = -inf gives 0 whatever the (then finite) reference; a nan score stays nan
            const float p0 = ex2(y[r] - (mm[r] == -INFINITY ? 0.f : mm[r]));
            const float p1 = ex2(y[r + 1] - (mm[r + 1] == -INFINITY ? 0.f : mm[r + 1]));
            ls[r] = fmaf(p0, iv, ls[r]);
            ls[r + 1] = fmaf(p1, iv, ls[r + 1]);
            float a = p0, b = p1;
#pragma unroll
            for (int j = 0; j < 3; ++j) {
              const uint32_t c = e4m3x2(a, b);
              pb[swz(j * R + r, k)] = uint8_t(c);
              pb[swz(j * R + r + 1, k)] = uint8_t(c >> 8);
              const float2 back = f16x2_to_f32x2(e4m3x2_to_f16x2(c));
              a = (a - back.x) * 16.f;
              b = (b - back.y) * 16.f;
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(&ctl->p_full[bsel]);
        }
        t_glob += n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->q_empty[n_items & 1]);
        // ---- epilogue: O^T of this item, the row sums over the 128 keys
        if (!mbar_wait(&ctl->o_full, n_items & 1, abort_flag)) return Run::kGaveUp;
        ++n_items;
        tc_fence_after();
        tmem_ldn<NO>(tmem + lane_off + kColO, ov);
        tc_fence_before();
        mbar_arrive(&ctl->o_free);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
          for (int r = 0; r < R; ++r) ls[r] += __shfl_xor_sync(0xffffffffu, ls[r], o);
        }
        if (lane == 0) {
#pragma unroll
          for (int r = 0; r < R; ++r) ctl->lsum[r][warp] = ls[r];
        }
        if (named_bar_leave(1, 128, false)) return Run::kTold;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 l4 = *reinterpret_cast<const float4*>(ctl->lsum[r]);
          ls[r] = (l4.x + l4.y) + (l4.z + l4.w);
        }
      }
      pdl_wait();   // outputs and partials may still be read by the previous kernel
      const int d = k;   // this thread's TMEM lane of O^T is column d of the output rows
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) continue;
        const float l = ls[r];
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float sum = fmaf(__uint_as_float(ov[2 * R + r]), 0.00390625f,
                               fmaf(__uint_as_float(ov[R + r]), 0.0625f, __uint_as_float(ov[r])));
        if (it.slot < 0) {
          const int64_t row = int64_t(it.q0 + r / G) * p.num_q_heads + it.g * G + r % G;
          p.o[row * kHeadDim + d] = __float2bfloat16_rn(sum * inv);
          if (d == r && p.row_lse)
            p.row_lse[row] = ((mm[r] == -INFINITY ? 0.f : mm[r]) + __log2f(l)) * 0.69314718055994531f;
        } else {
          float* dst = p.part + (size_t(it.slot) * p.item_rows + r) * kPartStride;
          reinterpret_cast<__half*>(dst)[d] = __float2half_rn(sum * inv);
          if (d == r) reinterpret_cast<float4*>(dst + kHeadDim / 2)[0] = make_float4(mm[r], l, 0.f, 0.f);
        }
      }
      return Run::kOn;
    };
    int bad = 0;
    Run run = Run::kOn;
    while (run == Run::kOn && kv8_take(&ctl->ring, n_it++, it, abort_flag, bad)) {
      const int n = it.n;
      const int R = pad_rows(it.n_q * G);   // at most 16 rows on this path
      run = R == 4   ? run_item(std::integral_constant<int, 4>{}, n)
            : R == 8 ? run_item(std::integral_constant<int, 8>{}, n)
                     : run_item(std::integral_constant<int, 16>{}, n);
    }
    if (run == Run::kGaveUp) bad = 1;
    if (bad) raise_abort(ctl, p.err);
    if (run != Run::kTold) named_bar_leave(1, 128, bad);
  } else if (warp == 4) {
    // ------------------------------------------------------------ producer
    uint32_t t_glob = 0, n_k = 0, n_v = 0;   // n_k, n_v: K and V tiles issued
    int bad = 0;
    Kv8Walk<true> walk;
    int cached_b = -1;
    kv8_line<true>(p, prefix, &ctl->ring, lane);
    walk.start(&ctl->ring);
    while (!bad && walk.next(p, prefix, &ctl->ring, it)) {
      if (!kv8_put(&ctl->ring, n_it++, it, lane, abort_flag)) { bad = 1; break; }
      const int n = it.n;
      const int sub = lane & 7;
      Kv8Pages<kPagesPerTile> pages;
      pages.start(p, walk.req, &ctl->chunks, walk.b != cached_b, it.t_begin, it.g, lane);
      cached_b = walk.b;
      for (int i = 0; i < n; ++i) {
        const uint32_t t = t_glob + i;
        const int wi = i % Kv8Pages<kPagesPerTile>::kTiles;
        if (wi == 0 && i > 0) pages.advance();
        const int from = wi * kPagesPerTile + sub;
        const int page = __shfl_sync(0xffffffffu, pages.cur.page, from);
        const int nvalid = __shfl_sync(0xffffffffu, pages.cur.nvalid, from);
        const int lstart = __shfl_sync(0xffffffffu, pages.cur.lstart, from);
        // the boxes first: they need the page alone, the descriptor its scales
        const int box = page >= 0 ? ((p.layer * p.num_pages + page) * p.num_kv_heads + it.g) * kPage
                                      : -kPage;   // fully out of range: the box is zero-filled
        const int s = t % kKSt;
        if (t >= uint32_t(kKSt) && !mbar_wait(&ctl->kempty[s], ((t / kKSt) - 1) & 1, abort_flag)) { bad = 1; break; }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&ctl->kfull[s], kTile8);
        __syncwarp();
        if (lane < 8) tma_load_2d(sK + s * kTile8 + sub * kPageBytes8, &tm_k, &ctl->kfull[s], 0, box);
        ++n_k;
        const uint32_t slot = t % kDescSlots;
        if (t >= kDescSlots && !mbar_wait(&ctl->desc_empty[slot], ((t / kDescSlots) - 1) & 1, abort_flag)) {
          bad = 1;
          break;
        }
        TileDesc* d = &ctl->desc[slot];
        if (wi == 0) pages.settle(p);
        const float ks = __shfl_sync(0xffffffffu, pages.cur_k, from), vs = __shfl_sync(0xffffffffu, pages.cur_v, from);
        if (lane < 8) {
          d->ks[sub] = ks;
          d->lstart[sub] = lstart;
          d->nvalid[sub] = uint8_t(nvalid);
        } else if (lane < 16) {
          d->lv[sub] = __log2f(vs);
          d->iv[sub] = __frcp_rn(vs);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->desc_full[slot]);
        const int sv = t % kVSt;
        if (t >= uint32_t(kVSt) && !mbar_wait(&ctl->vempty[sv], ((t / kVSt) - 1) & 1, abort_flag)) { bad = 1; break; }
        if (lane >= 8 && lane < 16) ctl->vnv[sv][sub] = uint8_t(nvalid);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&ctl->vfull[sv], kTile8);
        __syncwarp();
        if (lane >= 8 && lane < 16) tma_load_2d(sV + sv * kTile8 + sub * kPageBytes8, &tm_v, &ctl->vfull[sv], 0, box);
        ++n_v;
        if (wi == 0) pages.ahead(p, walk.req, &ctl->chunks, i, it.g, lane);
      }
      t_glob += n;
    }
    it.n = 0;
    if (!bad && !kv8_put(&ctl->ring, n_it, it, lane, abort_flag)) bad = 1;
    if (p.part) {
      pdl_wait();   // the previous call's combine may still read the cuts
      if (lane == 0) p.cuts[blockIdx.x] = walk.cut;
    }
    if (bad) raise_abort(ctl, p.err);
    // Let every copy this warp issued land before the CTA exits, whether a role
    // has given up by now or does so later. (They have landed, or the others
    // still wait for them: it costs nothing.)
    if (lane == 0) {
      for (uint32_t t = n_k > kKSt ? n_k - kKSt : 0; t < n_k; ++t) wait_quiet(&ctl->kfull[t % kKSt], (t / kKSt) & 1);
      for (uint32_t t = n_v > kVSt ? n_v - kVSt : 0; t < n_v; ++t) wait_quiet(&ctl->vfull[t % kVSt], (t / kVSt) & 1);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------------------------ V slots without a token -> 0
    uint32_t t_glob = 0;
    int bad = 0;
    while (!bad && kv8_take(&ctl->ring, n_it++, it, abort_flag, bad)) {
      const int n = it.n;
      for (int i = 0; i < n; ++i) {
        const uint32_t t = t_glob + i;
        const int sv = t % kVSt;
        if (!mbar_wait(&ctl->vfull[sv], (t / kVSt) & 1, abort_flag)) { bad = 1; break; }
        const uint2 nv = *reinterpret_cast<const uint2*>(ctl->vnv[sv]);
        if (nv.x != 0x10101010u || nv.y != 0x10101010u) {
          for (int u = lane; u < kBN * 8; u += 32) {   // 16-byte vectors of the tile's rows
            const int row = u >> 3;
            if ((row & 15) >= int(ctl->vnv[sv][row >> 4]))
              *reinterpret_cast<uint4*>(sV + sv * kTile8 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->vready[sv]);
      }
      t_glob += n;
    }
    if (bad) raise_abort(ctl, p.err);
    __syncwarp();
  } else if (warp == 7) {
    // ------------------------------------------------------------ queries, one item ahead
    const int c = lane & 7;   // 16 channels: 16c .. 16c + 15
    uint32_t q_iter = 0;
    int bad = 0;
    pdl_wait();               // q may be the previous kernel's output
    while (!bad && kv8_take(&ctl->ring, n_it++, it, abort_flag, bad)) {
      const int rows = it.n_q * G, R = pad_rows(rows);
      const int buf = int(q_iter & 1u);
      if (q_iter >= 2 && !mbar_wait(&ctl->q_empty[buf], ((q_iter >> 1) - 1) & 1, abort_flag)) { bad = 1; break; }
      uint8_t* dst = sQ + buf * kQBytes;
      for (int r0 = 0; r0 < R; r0 += 4) {
        const int r = r0 + (lane >> 3);
        uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (r < rows) {
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + ((int64_t(it.q0) + r / G) * p.num_q_heads + it.g * G + r % G) * kHeadDim + 16 * c);
          v[0] = src[0];
          v[1] = src[1];
        }
        QuerySplit q;
        q.split(v[0], v[1], lane, 16.f);
        *reinterpret_cast<uint4*>(dst + swz(r, 16 * c)) = q.hi;
        *reinterpret_cast<uint4*>(dst + swz(R + r, 16 * c)) = q.lo;
        if (c == 0) ctl->sq[buf][r] = q.scale * p.scale_log2;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[buf]);
      ++q_iter;
    }
    if (bad) raise_abort(ctl, p.err);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ MMA issuer (warp 5)
    {
      const uint32_t leader = elect_one();
      const uint32_t k_lo0 = sdesc_lo(smem_u32(sK), 16), v_lo0 = sdesc_lo(smem_u32(sV), 0);
      const uint32_t q_lo0 = sdesc_lo(smem_u32(sQ), 16), p_lo0 = sdesc_lo(smem_u32(sP), 16);
      uint32_t t_glob = 0, n_items = 0;
      int bad = 0;
      while (!bad && kv8_take(&ctl->ring, n_it++, it, abort_flag, bad)) {
        const int n = it.n;
        const int R = pad_rows(it.n_q * G);
        const uint32_t idesc_qk = idesc_e4m3_f32(kBN, uint32_t(n_qk(R)), 0, 0);
        const uint32_t idesc_pv = idesc_e4m3_f32(kHeadDim, uint32_t(n_pv(R)), 1, 0);
        const int qb = int(n_items & 1u);
        const uint32_t q_lo = q_lo0 + qb * (kQBytes >> 4);
        if (!mbar_wait(&ctl->q_full[qb], (n_items >> 1) & 1, abort_flag)) { bad = 1; break; }
        tc_fence_after();
        // S^T of tile j of the item into buffer (tile parity)
        auto qk = [&](int j) {
          const uint32_t t = t_glob + j;
          const int s = t % kKSt;
          if (!mbar_wait(&ctl->kfull[s], (t / kKSt) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint32_t k_lo = k_lo0 + s * (kTile8 >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_f8(leader, tmem + 32u * (t & 1u), k_lo + 2 * kk, q_lo + 2 * kk, idesc_qk, kk > 0);
          tc_commit_by(leader, &ctl->s_full[t & 1]);
          tc_commit_by(leader, &ctl->kempty[s]);
          if (j == n - 1) tc_commit_by(leader, &ctl->q_empty[qb]);   // the rest of the item reads no Q
          return true;
        };
        for (int j = 0; j < n && j < 2 && !bad; ++j)
          if (!qk(j)) bad = 1;
        for (int i = 0; i < n && !bad; ++i) {
          const uint32_t t = t_glob + i;
          const int sv = t % kVSt;
          const int bsel = int(t & 1u);
          if (!mbar_wait(&ctl->vready[sv], (t / kVSt) & 1, abort_flag)) { bad = 1; break; }
          if (i == 0 && n_items > 0 && !mbar_wait(&ctl->o_free, (n_items - 1) & 1, abort_flag)) { bad = 1; break; }
          if (!mbar_wait(&ctl->p_full[bsel], (t >> 1) & 1, abort_flag)) { bad = 1; break; }
          tc_fence_after();
          const uint32_t v_lo = v_lo0 + sv * (kTile8 >> 4), p_lo = p_lo0 + bsel * (kPBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_f8(leader, tmem + kColO, v_lo + kk * (32 * 128 >> 4), p_lo + 2 * kk, idesc_pv, (i > 0) || (kk > 0));
          tc_commit_by(leader, &ctl->pv_done[bsel]);
          tc_commit_by(leader, &ctl->vempty[sv]);
          if (i == n - 1) tc_commit_by(leader, &ctl->o_full);
          if (i + 2 < n && !qk(i + 2)) { bad = 1; break; }
        }
        if (bad) break;
        t_glob += n;
        ++n_items;
      }
      if (bad) raise_abort(ctl, p.err);
      tc_commit_by(leader, &ctl->teardown);
      wait_quiet(&ctl->teardown, 0);
    }
    __syncwarp();
  }

  pdl_wait();   // the grid completes only after the kernel before it, items or none
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

cudaError_t launch_kv8_decode(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p, int grid,
                              cudaStream_t stream) {
  const size_t smem = 1024 + d8::kSmemData + sizeof(d8::Ctrl) + sizeof(int32_t) * (p.batch.num_requests + 1) + 64;
  static SmemAttr attr;
  cudaError_t e = ensure_smem_attr(kv8_decode_kernel, attr, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_decode_kernel, dim3(grid), dim3(d8::kThreads), smem, stream, 1, tk, tv, p);
}

}  // namespace rag
