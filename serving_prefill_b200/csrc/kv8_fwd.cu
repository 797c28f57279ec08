// Attention of a request's query tokens over its pages of the 8-bit pool
// (TurboRAG page, "Technical Details": softmax(Q K^T / sqrt(d_k) + M) V over
// the concatenated cache; here the cache holds e4m3 codes, value = code *
// scale of the page and KV head, and the query tokens' own keys were appended
// to it).
//
// One persistent CTA per SM walks its stretch of the work units (request, KV head,
// two 128-row Q tiles; their key tiles); a row is (query token, head in the group),
// 128 / G tokens to a tile. The scores come from the codes themselves:
//   q = s_q (hi + lo), hi and lo e4m3, s_q a power of two per row, split once
//       by kv8_split_q_kernel: a bf16 value's 8 significant bits are two e4m3
//       significands, so hi + lo is the value itself from s_q / 4 on, where lo's
//       last bit is e4m3's smallest step, 2^-9 s_q; that is at least from 2^-9 of
//       the row's largest on, and smaller values are off by at most 2^-10 s_q,
//       2^-17 of the largest
//   S = hi K8 + lo K8: two kind::f8f6f4 products of twice the 16-bit rate, so
//       they cost what one bf16 product would, K tiles go from TMA to the
//       tensor core untouched, and no page is converted for the scores
//   score = S * (s_q * scale of the page): one factor per row and page, folded
//       into the softmax's multiply-add
// V enters as fp16 (code * scale, exact for power-of-two scales from 2^-15 on;
// below, fp16's smallest step is coarser than the code's, and the value is off by
// at most 2^-25; another scale is itself rounded to fp16 first, as rounding the
// product instead made the conversion the slowest role: 147 us against 133 for
// the 16 prompts):
// weights in e4m3 would lose what the softmax kept, and splitting them costs
// the issue-bound softmax warps more than two converting warps cost.
//   producer warp : per tile 5 + 5 TMA page boxes of 2 KB (K, V), the scales
//                   (loaded a tile ahead), the mask descriptor; the items
//   MMA warp      : S_i = Q_i K8^T for both Q tiles, then O_i += P_i V
//   2 convert warps: V codes -> fp16 in the 128-byte swizzle, slots that hold
//                   no token zeroed
//   2 x 4 softmax warps: thread = row = TMEM lane; mask, online max and sum in
//                   the log2 domain, P (fp16) to columns of its own
// A tile is 80 keys: then S and P of both Q tiles have tensor-memory columns of
// their own beside the two O (2 * 80 + 2 * 40 + 2 * 128 = 496 of 512), and S of
// the next tile is computed as soon as this one is in registers, under its
// exponentials. With 128 keys P has to lie over S and every tile pays the round
// trip softmax -> PV -> QK -> softmax, but there are fewer of them. Measured
// (128 / 80 keys): 506 / 530 us for 256 tokens of 64 heads over 65,792 keys,
// 156 / 148 us for 16 prompts over ragged chunks, 41.3 / 41.8 us for 100 tokens
// over 10,100 keys. 80 is kept: the ragged case is the usual one, and the
// softmax warps hardly spill. (With later steps the 80-key form takes 507, 133
// and 41 us.)
// What bounds it: a tile of two Q tiles takes 2,700 cycles, of which the tensor
// core is busy 1,450 (QK at N = 80 is bound by shared-memory reads of its
// operands, 52 cycles a product against 40) and the exponential unit 1,280; with
// exponentials, conversion and most products taken out of a copy it still takes
// 1,900, so the rest is the chain of hand-offs between the roles.
// Every wait is bounded; a timeout raises a device error instead of hanging.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv8.cuh"
#include "params.cuh"

namespace rag {
namespace f8 {

constexpr int kPages = kFwdPages;                // pages of a key tile
constexpr int kKeys = kPages * kPage;            // keys of a tile
constexpr int kKSt = 4;                          // K stages (codes)
constexpr int kRSt = 3;                          // V stages (codes)
constexpr int kVSt = 3;                          // V stages (fp16)
constexpr int kDescSlots = 4;
constexpr int kPart8 = kBM * kHeadDim;           // hi or lo part of a Q tile
constexpr int kQTileBytes = 2 * kPart8;
constexpr int kKTile = kKeys * kHeadDim;         // K or V codes
constexpr int kVTile = kKeys * kHeadDim * 2;     // fp16
constexpr int kVHalf = kVTile / 2;               // 64 columns of d
constexpr int kThreads = 384;                    // 8 softmax + producer, MMA, 2 convert warps
constexpr float kRescale = 8.0f;                 // log2 units: rescale O when the max grows by > 2^8

// TMEM columns: S_i, P_i (fp16 pairs), O_i
__host__ __device__ constexpr uint32_t col_s(int qt) { return uint32_t(kKeys) * qt; }
__host__ __device__ constexpr uint32_t col_p(int qt) { return 2u * kKeys + uint32_t(kKeys / 2) * qt; }
__host__ __device__ constexpr uint32_t col_o(int qt) { return 256u + 128u * qt; }
static_assert(col_p(kQTiles) <= 256, "tensor memory");

struct TileDesc {
  float ks[kPages];
  int32_t lstart[kPages];   // logical position of the page's slot 0
  int32_t nvalid[kPages];
  int32_t full;             // every slot of the pages is a token
  int32_t max_pos;          // largest logical position of the tile
};
struct VInfo {
  float vs[kPages];
  int32_t nvalid[kPages];
};

struct Ctrl {
  uint64_t q_full, q_empty;
  uint64_t kfull[kKSt], kempty[kKSt];
  uint64_t rfull[kRSt], rempty[kRSt];
  uint64_t vfull[kVSt], vempty[kVSt];
  uint64_t s_full[kQTiles], s_free[kQTiles], p_full[kQTiles], pv_done[kQTiles], o_full[kQTiles], o_free[kQTiles];
  uint64_t teardown;
  uint64_t desc_full[kDescSlots], desc_empty[kDescSlots];
  TileDesc desc[kDescSlots];
  VInfo vinfo[kRSt];
  ChunkCache chunks;
  Kv8Ring ring;
  uint32_t tmem_base;
  int32_t abort;
};

constexpr size_t kSmemData = size_t(kQTiles) * kQTileBytes + size_t(kKSt + kRSt) * kKTile + size_t(kVSt) * kVTile;
constexpr size_t smem_bytes(int num_requests) {
  return 1024 + kSmemData + sizeof(Ctrl) + sizeof(int32_t) * (size_t(num_requests) + 1);
}
static_assert(smem_bytes(kMaxRequests) <= 227 * 1024, "shared memory of a CTA");

// 32 lanes x 16 columns of 32-bit: thread i of the warp gets lane (base + i).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// The 40 columns of a tile's P.
__device__ __forceinline__ void tmem_st_p(uint32_t taddr, const uint32_t (&r)[kKeys / 2]) {
  static_assert(kKeys / 2 == 40, "16 + 16 + 8 columns");
  tmem_st16(taddr, r);
  tmem_st16(taddr + 16, r + 16);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr + 32), "r"(r[32]),
               "r"(r[33]), "r"(r[34]), "r"(r[35]), "r"(r[36]), "r"(r[37]), "r"(r[38]), "r"(r[39])
               : "memory");
}

// Low words of the operands' descriptors. Q parts and K tiles are K-major rows
// of 128 codes: a k-step of 32 codes is 32 bytes on (2 in units of 16). A V tile
// [80 keys][128 d] fp16 is the B operand with N = d contiguous: a k-step of 16
// keys is 2 KB on, the two 64-wide halves of d are 10 KB apart (leading offset).

}  // namespace f8

using namespace f8;

__global__ void __launch_bounds__(f8::kThreads, 1)
kv8_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const Kv8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + kQTiles * kQTileBytes;
  uint8_t* sR = sK + kKSt * kKTile;
  uint8_t* sV = sR + kRSt * kKTile;
  Ctrl* ctl = reinterpret_cast<Ctrl*>(sV + kVSt * kVTile);
  int32_t* prefix = reinterpret_cast<int32_t*>(ctl + 1);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int G = p.group;
  const int TT = p.toks_per_block / kQTiles;   // query tokens of a Q tile

  pdl_launch_dependents();

  if (tid == 0) {
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->q_empty, 1);
    for (int s = 0; s < kKSt; ++s) { mbar_init(&ctl->kfull[s], 1); mbar_init(&ctl->kempty[s], 1); }
    for (int s = 0; s < kRSt; ++s) { mbar_init(&ctl->rfull[s], 1); mbar_init(&ctl->rempty[s], 2); }
    for (int s = 0; s < kVSt; ++s) { mbar_init(&ctl->vfull[s], 2); mbar_init(&ctl->vempty[s], 1); }
    for (int q = 0; q < kQTiles; ++q) {
      mbar_init(&ctl->s_full[q], 1);
      mbar_init(&ctl->s_free[q], 128);
      mbar_init(&ctl->p_full[q], 128);
      mbar_init(&ctl->pv_done[q], 1);
      mbar_init(&ctl->o_full[q], 1);
      mbar_init(&ctl->o_free[q], 128);
    }
    mbar_init(&ctl->teardown, 1);
    for (int s = 0; s < kDescSlots; ++s) {
      mbar_init(&ctl->desc_full[s], 1);
      mbar_init(&ctl->desc_empty[s], 8);   // one arrival per softmax warp
    }
    kv8_ring_init(&ctl->ring, 11);   // 8 softmax warps, MMA, 2 convert warps
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) { tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  volatile int* abort_flag = &ctl->abort;
  Kv8Item it = {};
  uint32_t n_it = 0;   // items taken

  // The pool and the batch are read at once; the split queries, which the
  // kernel before this one writes, and every output only after pdl_wait.
  // registers: the softmax warpgroups take 208 per thread, the four role warps 88
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
    // ------------------------------------------------------------ softmax warpgroup qt
    const int qt = warp >> 2;
    const int r = tid & 127;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_off + col_o(qt);
    uint32_t t_glob = 0;   // tiles seen by the CTA
    uint32_t n_s = 0;      // tiles of this Q tile so far (S read, P written, PV issued)
    uint32_t n_of = 0;     // items whose O_qt has been read
    int bad = 0;
    pdl_wait();            // the row scales come from the kernel before this one
    while (!bad && kv8_take(&ctl->ring, n_it++, it, abort_flag, bad)) {
      const int n = it.n;
      const int tok0 = it.rb * p.toks_per_block;
      const bool active = qt == 0 || it.n_q - tok0 > TT;   // Q tile 1 may hold no row
      const int tok = tok0 + qt * TT + r / G;
      const int head = it.g * G + r % G;
      const bool row_valid = active && r < TT * G && tok < it.n_q;
      const int64_t row = int64_t(it.q0 + tok) * p.num_q_heads + head;
      const int lim = p.causal ? it.n_doc - it.n_q + tok : it.n_doc - 1;   // last visible position
      const float c_row = row_valid ? p.scale_log2 * __ldcg(p.qscale + row) : 0.f;
      const bool warp_live = __any_sync(0xffffffffu, row_valid);
      float m_ref = -INFINITY, l_sum = 0.f;
      for (int i = 0; i < n; ++i) {
        const uint32_t t = t_glob + i;
        const uint32_t slot = t % kDescSlots;
        if (!mbar_wait(&ctl->desc_full[slot], (t / kDescSlots) & 1, abort_flag)) { bad = 1; break; }
        const TileDesc* td = &ctl->desc[slot];
        float cp[kPages];
        int nv[kPages];   // slots of each page that this row sees
        const int max_pos = td->max_pos;
        const bool masked = !td->full || max_pos > lim;
#pragma unroll
        for (int g = 0; g < kPages; ++g) {
          cp[g] = c_row * td->ks[g];
          nv[g] = kPage;
        }
        if (masked) {
#pragma unroll
          for (int g = 0; g < kPages; ++g) nv[g] = min(td->nvalid[g], lim - td->lstart[g] + 1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->desc_empty[slot]);
        if (!active) continue;
        const uint32_t s_addr = tmem + lane_off + col_s(qt);
        if (!mbar_wait(&ctl->s_full[qt], n_s & 1, abort_flag)) { bad = 1; break; }
        tc_fence_after();
        if (!warp_live) {
          // All 32 rows lie past the query block: every arrival, no work. An
          // arrival for P waits, as the other warps' does, for PV of the tile
          // before: S of the next tile may be there already, and an arrival
          // for it must not count for this one.
          mbar_arrive(&ctl->s_free[qt]);
          if (i > 0 && !mbar_wait(&ctl->pv_done[qt], (n_s - 1) & 1, abort_flag)) { bad = 1; break; }
          mbar_arrive(&ctl->p_full[qt]);
          ++n_s;
          continue;
        }
        float x[kKeys];
        {
          uint32_t u0[32], u1[32], u2[16];
          tmem_ld32(s_addr + 0, u0);
          tmem_ld32(s_addr + 32, u1);
          tmem_ld16(s_addr + 64, u2);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            x[j] = __uint_as_float(u0[j]);
            x[32 + j] = __uint_as_float(u1[j]);
            if (j < 16) x[64 + j] = __uint_as_float(u2[j]);
          }
        }
        // S is in registers: the next tile's product may overwrite it
        tc_fence_before();
        mbar_arrive(&ctl->s_free[qt]);
        if (masked) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if ((c & 15) >= nv[c >> 4]) x[c] = -INFINITY;
        }
        // row max: the largest raw score of each page, scaled by its factor (> 0)
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < kPages; ++g) {
          const float* xg = x + 16 * g;
          float a = fmax3(xg[0], xg[1], xg[2]), b = fmax3(xg[3], xg[4], xg[5]);
          a = fmax3(a, xg[6], xg[7]);
          b = fmax3(b, xg[8], xg[9]);
          a = fmax3(a, xg[10], xg[11]);
          b = fmax3(b, xg[12], xg[13]);
          a = fmax3(a, xg[14], xg[15]);
          mx = fmaxf(mx, fmaxf(a, b) * cp[g]);
        }
        // PV of the previous tile has read P (and added to O)
        if (i > 0 && !mbar_wait(&ctl->pv_done[qt], (n_s - 1) & 1, abort_flag)) { bad = 1; break; }
        float alpha = 1.f;
        bool need = false;
        if (i == 0) {
          m_ref = mx;
        } else if (mx > m_ref + kRescale) {
          alpha = ex2(m_ref - mx);
          need = true;
        }
        if (__any_sync(0xffffffffu, need)) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t u[32];
            tmem_ld32(o_addr + 32 * c, u);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * alpha);
            tmem_st32(o_addr + 32 * c, u);
          }
          tmem_wait_st();
          if (need) { l_sum *= alpha; m_ref = mx; }
        }
        const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
        const float2 nm2 = make_float2(neg_m, neg_m);
        float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
        uint32_t pk[kKeys / 2];
#pragma unroll
        for (int j = 0; j < kKeys / 2; ++j) {
          const float c = cp[j >> 3];
          const float2 y = ffma2(make_float2(x[2 * j], x[2 * j + 1]), make_float2(c, c), nm2);
          const float2 e = make_float2(ex2(y.x), ex2(y.y));
          ls[j & 3] = fadd2(ls[j & 3], e);
          pk[j] = pack_f16x2(e.x, e.y);
        }
        tmem_st_p(tmem + lane_off + col_p(qt), pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&ctl->p_full[qt]);
        const float2 ls01 = fadd2(ls[0], ls[1]), ls23 = fadd2(ls[2], ls[3]);
        l_sum += (ls01.x + ls01.y) + (ls23.x + ls23.y);
        ++n_s;
      }
      if (bad) break;
      t_glob += n;
      if (!active) continue;

      // ---- epilogue: O of this Q tile
      // the MMA warp commits o_full once per item after the item's last PV
      if (!mbar_wait(&ctl->o_full[qt], n_of & 1, abort_flag)) { bad = 1; break; }
      ++n_of;
      tc_fence_after();
      if (!warp_live) {   // no row of this warp is read or written
        tc_fence_before();
        mbar_arrive(&ctl->o_free[qt]);
        continue;
      }
      float o[kHeadDim];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t u[32];
        tmem_ld32(o_addr + 32 * c, u);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[32 * c + j] = __uint_as_float(u[j]);
      }
      tc_fence_before();
      mbar_arrive(&ctl->o_free[qt]);
      // l = 0: the row saw no key of this item; a row of nan (a nan query) keeps it
      const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
      if (!row_valid) continue;
      if (it.slot < 0) {
        uint4* dst = reinterpret_cast<uint4*>(p.o + row * kHeadDim);
#pragma unroll
        for (int c = 0; c < kHeadDim / 8; ++c) {
          uint4 v;
          v.x = pack_bf16x2(o[8 * c + 0] * inv, o[8 * c + 1] * inv);
          v.y = pack_bf16x2(o[8 * c + 2] * inv, o[8 * c + 3] * inv);
          v.z = pack_bf16x2(o[8 * c + 4] * inv, o[8 * c + 5] * inv);
          v.w = pack_bf16x2(o[8 * c + 6] * inv, o[8 * c + 7] * inv);
          dst[c] = v;
        }
        const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
        if (p.row_lse) p.row_lse[row] = (m_use + __log2f(l_sum)) * 0.69314718055994531f;
      } else {
        // partial row: this piece's own softmax average O/l in fp16 (|O/l| is
        // bounded by max |V|), then its reference max m and sum l in fp32
        uint4* dst = reinterpret_cast<uint4*>(p.part + (size_t(it.slot) * p.item_rows + qt * kBM + r) * kPartStride);
#pragma unroll
        for (int c = 0; c < kHeadDim / 8; ++c) {
          uint4 v;
          v.x = pack_f16x2(o[8 * c + 0] * inv, o[8 * c + 1] * inv);
          v.y = pack_f16x2(o[8 * c + 2] * inv, o[8 * c + 3] * inv);
          v.z = pack_f16x2(o[8 * c + 4] * inv, o[8 * c + 5] * inv);
          v.w = pack_f16x2(o[8 * c + 6] * inv, o[8 * c + 7] * inv);
          dst[c] = v;
        }
        reinterpret_cast<float4*>(dst + kHeadDim / 8)[0] = make_float4(m_ref, l_sum, 0.f, 0.f);
      }
    }
    if (bad) raise_abort(ctl, p.err);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
    if (warp == 8) {
      // ------------------------------------------------------------ producer
      uint32_t t_glob = 0, n_k = 0, n_v = 0;   // n_k, n_v: K and V tiles issued
      int bad = 0;
      Kv8Walk<false> walk;
      int cached_b = -1;
      kv8_line<false>(p, prefix, &ctl->ring, lane);
      walk.start(&ctl->ring);
      while (!bad && walk.next(p, prefix, &ctl->ring, it)) {
        if (!kv8_put(&ctl->ring, n_it++, it, lane, abort_flag)) { bad = 1; break; }
        const int n = it.n;
        const int sub = lane & 7;
        const bool mine = lane < 16 && sub < kPages;   // a page of K (lanes 0-7) or of V (lanes 8-15)
        Kv8Pages<kPages> pages;
        pages.start(p, walk.req, &ctl->chunks, walk.b != cached_b, it.t_begin, it.g, lane);
        cached_b = walk.b;
        for (int i = 0; i < n; ++i) {
          const uint32_t t = t_glob + i;
          const int wi = i % Kv8Pages<kPages>::kTiles;
          if (wi == 0 && i > 0) pages.advance();
          const int from = wi * kPages + (mine ? sub : 0);
          const int page = __shfl_sync(0xffffffffu, pages.cur.page, from);
          const int nvalid = __shfl_sync(0xffffffffu, pages.cur.nvalid, from);
          const int lstart = __shfl_sync(0xffffffffu, pages.cur.lstart, from);
          const int box = page >= 0 ? ((p.layer * p.num_pages + page) * p.num_kv_heads + it.g) * kPage
                                    : -kPage;   // fully out of range: the box is zero-filled
          const int s = t % kKSt;
          if (t >= uint32_t(kKSt) && !mbar_wait(&ctl->kempty[s], ((t / kKSt) - 1) & 1, abort_flag)) { bad = 1; break; }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&ctl->kfull[s], kKTile);
          __syncwarp();
          if (mine && lane < 8) tma_load_2d(sK + s * kKTile + sub * kPageBytes8, &tm_k, &ctl->kfull[s], 0, box);
          ++n_k;
          // the K boxes need the page alone, what follows its scales
          if (wi == 0) pages.settle(p);
          const float ks = __shfl_sync(0xffffffffu, pages.cur_k, from), vs = __shfl_sync(0xffffffffu, pages.cur_v, from);
          const uint32_t slot = t % kDescSlots;
          if (t >= kDescSlots && !mbar_wait(&ctl->desc_empty[slot], ((t / kDescSlots) - 1) & 1, abort_flag)) {
            bad = 1;
            break;
          }
          TileDesc* d = &ctl->desc[slot];
          const unsigned full_pages = __ballot_sync(0xffffffffu, lane < kPages && nvalid == kPage);
          const int last = lane < kPages && nvalid > 0 ? lstart + nvalid - 1 : -1;
          const int max_pos = __reduce_max_sync(0xffffffffu, last);
          if (lane < kPages) {
            d->ks[lane] = ks;
            d->lstart[lane] = lstart;
            d->nvalid[lane] = nvalid;
          }
          if (lane == 0) { d->full = full_pages == (1u << kPages) - 1 ? 1 : 0; d->max_pos = max_pos; }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->desc_full[slot]);
          const int sv = t % kRSt;
          if (t >= uint32_t(kRSt) && !mbar_wait(&ctl->rempty[sv], ((t / kRSt) - 1) & 1, abort_flag)) { bad = 1; break; }
          if (mine && lane >= 8) {
            ctl->vinfo[sv].vs[sub] = vs;
            ctl->vinfo[sv].nvalid[sub] = nvalid;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&ctl->rfull[sv], kKTile);
          __syncwarp();
          if (mine && lane >= 8) tma_load_2d(sR + sv * kKTile + sub * kPageBytes8, &tm_v, &ctl->rfull[sv], 0, box);
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
        for (uint32_t t = n_v > kRSt ? n_v - kRSt : 0; t < n_v; ++t) wait_quiet(&ctl->rfull[t % kRSt], (t / kRSt) & 1);
      }
      __syncwarp();
    } else if (warp >= 10) {
      // ------------------------------------------------------------ convert warps
      // Each warp takes every other group of 4 keys. A lane reads 16 codes of
      // a row and writes two 16-byte vectors of fp16; lanes of the upper half
      // of d write theirs in the other order, so that eight lanes cover all
      // banks with each store. Warp 10 also loads an item's Q tiles, which the
      // kernel before this one makes: the producer warp never waits for it, so
      // K and V stream in while the queries are still being split.
      const int c = lane & 7;                         // 16 codes: columns 16c .. 16c + 15
      uint32_t t_glob = 0, q_iter = 0;
      int bad = 0;
      while (!bad && kv8_take(&ctl->ring, n_it++, it, abort_flag, bad)) {
        const int n = it.n;
        if (warp == 10) {
          if (q_iter > 0 && !mbar_wait(&ctl->q_empty, (q_iter - 1) & 1, abort_flag)) { bad = 1; break; }
          if (lane == 0) {
            pdl_wait();
            const int tok0 = it.rb * p.toks_per_block;
            const int n_qt = it.n_q - tok0 > TT ? 2 : 1;
            mbar_arrive_expect_tx(&ctl->q_full, n_qt * 2 * TT * G * kHeadDim);
            for (int q = 0; q < n_qt; ++q) {
              tma_load_3d(sQ + q * kQTileBytes, &tm_q, &ctl->q_full, 0, it.g * G, it.q0 + tok0 + q * TT);
              tma_load_3d(sQ + q * kQTileBytes + kPart8, &tm_q, &ctl->q_full, kHeadDim, it.g * G,
                          it.q0 + tok0 + q * TT);
            }
          }
          ++q_iter;
          __syncwarp();
        }
        for (int i = 0; i < n; ++i) {
          const uint32_t t = t_glob + i;
          const int sr = t % kRSt, sv = t % kVSt;
          if (!mbar_wait(&ctl->rfull[sr], (t / kRSt) & 1, abort_flag)) { bad = 1; break; }
          if (t >= uint32_t(kVSt) && !mbar_wait(&ctl->vempty[sv], ((t / kVSt) - 1) & 1, abort_flag)) { bad = 1; break; }
          const uint8_t* src = sR + sr * kKTile;
          uint8_t* dst = sV + sv * kVTile + (c >> 2) * kVHalf;
#pragma unroll 5
          for (int j = 0; j < kKeys / 8; ++j) {
            const int row = 8 * j + 4 * (warp - 10) + (lane >> 3);
            const int pgi = row >> 4;
            const bool live = (row & 15) < ctl->vinfo[sr].nvalid[pgi];
            const __half2 sc = __float2half2_rn(ctl->vinfo[sr].vs[pgi]);
            uint4 u = *reinterpret_cast<const uint4*>(src + row * 128 + ((c ^ (row & 7)) << 4));
            if (!live) u = make_uint4(0u, 0u, 0u, 0u);
            uint32_t h[8];
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              h[2 * k] = e4m3x2_to_f16x2(uw[k] & 0xffffu);
              h[2 * k + 1] = e4m3x2_to_f16x2(uw[k] >> 16);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&h[k]), sc);
              h[k] = *reinterpret_cast<const uint32_t*>(&y);
            }
            const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
            const int k0 = 2 * (c & 3), first = c >> 2;       // chunks k0, k0 + 1 of the 64-column half
            uint8_t* d = dst + row * 128;
            *reinterpret_cast<uint4*>(d + (((k0 + first) ^ (row & 7)) << 4)) = first ? hi : lo;
            *reinterpret_cast<uint4*>(d + (((k0 + 1 - first) ^ (row & 7)) << 4)) = first ? lo : hi;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&ctl->vfull[sv]);
            mbar_arrive(&ctl->rempty[sr]);
          }
        }
        t_glob += n;
      }
      if (bad) raise_abort(ctl, p.err);
      if (lane == 0 && q_iter > 0) wait_quiet(&ctl->q_full, (q_iter - 1) & 1);
      __syncwarp();
    } else {
      // ------------------------------------------------------------ MMA issuer (warp 9)
      {
        const uint32_t leader = elect_one();
        const uint32_t idesc_qk = idesc_e4m3_f32(kBM, kKeys, 0, 0);
        const uint32_t idesc_pv = idesc_f16_f32(kBM, kHeadDim, 1);
        const uint32_t q_lo = sdesc_lo(smem_u32(sQ), 16);
        const uint32_t k_lo0 = sdesc_lo(smem_u32(sK), 16), v_lo0 = sdesc_lo(smem_u32(sV), kVHalf);
        uint32_t t_glob = 0, q_iter = 0;
        uint32_t n_s[kQTiles] = {0, 0};      // tiles done, per Q tile
        uint32_t n_item[kQTiles] = {0, 0};   // items begun, per Q tile
        int bad = 0;
        while (!bad && kv8_take(&ctl->ring, n_it++, it, abort_flag, bad)) {
          const int n = it.n;
          const int n_qt = it.n_q - it.rb * p.toks_per_block > TT ? 2 : 1;
          if (!mbar_wait(&ctl->q_full, q_iter & 1, abort_flag)) { bad = 1; break; }
          tc_fence_after();
          const bool two = n_qt == 2;
          // S_q = (hi + lo) K^T of tile j, once the softmax holds the S before
          // it in registers
          auto qk = [&](int q, int j) {
            const uint32_t t = t_glob + j;
            const int s = t % kKSt;
            if (!mbar_wait(&ctl->kfull[s], (t / kKSt) & 1, abort_flag)) return false;
            const uint32_t before = n_s[q] + j;   // reads of S_q by then
            if (before > 0 && !mbar_wait(&ctl->s_free[q], (before - 1) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t k_lo = k_lo0 + s * (kKTile >> 4), a_lo = q_lo + q * (kQTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss_f8(leader, tmem + col_s(q), a_lo + 2 * kk, k_lo + 2 * kk, idesc_qk, kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss_f8(leader, tmem + col_s(q), a_lo + (kPart8 >> 4) + 2 * kk, k_lo + 2 * kk, idesc_qk, 1);
            tc_commit_by(leader, &ctl->s_full[q]);
            if (q == n_qt - 1) {                  // the last read of this K stage
              tc_commit_by(leader, &ctl->kempty[s]);
              if (j == n - 1) tc_commit_by(leader, &ctl->q_empty);   // the rest of the item reads no Q
            }
            return true;
          };
          // O_q += P_q V of tile j
          auto pv = [&](int q, int j) {
            const uint32_t t = t_glob + j;
            const int sv = t % kVSt;
            if (!mbar_wait(&ctl->vfull[sv], (t / kVSt) & 1, abort_flag)) return false;
            if (j == 0) {
              if (n_item[q] > 0 && !mbar_wait(&ctl->o_free[q], (n_item[q] - 1) & 1, abort_flag)) return false;
              ++n_item[q];
            }
            if (!mbar_wait(&ctl->p_full[q], (n_s[q] + j) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t v_lo = v_lo0 + sv * (kVTile >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_ts_f16(leader, tmem + col_o(q), tmem + col_p(q) + kk * 8, v_lo + kk * (16 * 128 >> 4), idesc_pv,
                         (j > 0) || (kk > 0));
            tc_commit_by(leader, &ctl->pv_done[q]);
            if (j == n - 1) tc_commit_by(leader, &ctl->o_full[q]);
            if (q == n_qt - 1) tc_commit_by(leader, &ctl->vempty[sv]);   // the last read of this V stage
            return true;
          };
          // Q tile 1 follows Q tile 0 by about half a tile: its PV waits for Q
          // tile 0's next S, so that one warpgroup's exponentials run while the
          // other one's S and O are made. (Issued tile by tile for both, the
          // warpgroups run in step and share the exponential unit: 176 against
          // 162 us on 16 prompts, in a version with both otherwise alike.)
          if (!qk(0, 0)) bad = 1;
          for (int i = 0; i <= n && !bad; ++i) {
            if (two && i < n && !qk(1, i)) { bad = 1; break; }
            if (i + 1 < n && !qk(0, i + 1)) { bad = 1; break; }
            if (two && i > 0 && !pv(1, i - 1)) { bad = 1; break; }
            if (i < n && !pv(0, i)) { bad = 1; break; }
          }
          if (bad) break;
          for (int q = 0; q < n_qt; ++q) n_s[q] += n;
          t_glob += n;
          ++q_iter;
        }
        if (bad) raise_abort(ctl, p.err);
        // every MMA issued so far completes before TMEM is released
        tc_commit_by(leader, &ctl->teardown);
        wait_quiet(&ctl->teardown, 0);
      }
      __syncwarp();
    }
  }

  pdl_wait();   // the grid completes only after the kernel before it, items or none
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Queries as two e4m3 parts under a power-of-two scale per row: hi = e4m3(q /
// s), lo = e4m3(q / s - hi), s the smallest power of two with |q| <= 448 s.
// Eight lanes a row; the parts go to [row][hi 128 B, lo 128 B].
__global__ void __launch_bounds__(256) kv8_split_q_kernel(const Kv8Params p, int64_t rows) {
  pdl_launch_dependents();
  const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> 3;
  const int c = threadIdx.x & 7;
  const int64_t at = row < rows ? row : rows - 1;
  const uint4* src = reinterpret_cast<const uint4*>(p.q + at * kHeadDim + 16 * c);
  pdl_wait();   // q may be the previous kernel's output, and its attention may still read the split queries
  QuerySplit q;
  q.split(src[0], src[1], threadIdx.x & 31, 1.f);
  if (row >= rows) return;
  uint8_t* dst = p.qs + row * (2 * kHeadDim) + 16 * c;
  *reinterpret_cast<uint4*>(dst) = q.hi;
  *reinterpret_cast<uint4*>(dst + kHeadDim) = q.lo;
  if (c == 0) p.qscale[row] = q.scale;
}

// Merge the partial rows (O, m, l) of every cut unit:
//   m = max_s m_s, l = sum_s l_s 2^(m_s - m), O = sum_s O_s l_s 2^(m_s - m) / l.
// Block (c, y) merges 16 kPairs rows of the unit whose second piece CTA c left
// (nothing for other CTAs); a warp takes two rows at a time, 16 lanes each, a
// lane 8 of the 128 columns; lane j of a row holds the statistics of piece
// s0 + j, and the O slices of kBatch pieces are requested before any is used.
// Stretches leave two or three pieces a unit (4 at a time), pieces up to a
// dozen (8 at a time). Bound by its instructions per row: with a row to a warp
// 16 requests of 32-128 tokens took 139.9 us in all, so 136.3; a decode step is
// the same either way.
template <int kBatch, int kPairs, int kBlocks>
__global__ void __launch_bounds__(256, kBlocks) kv8_combine_kernel(const Kv8Params p) {
  constexpr int kRows = 16 * kPairs;
  pdl_launch_dependents();
  pdl_wait();   // partials and cuts come from the attention kernel
  const int row_in = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const int4 c4 = __ldcg(reinterpret_cast<const int4*>(p.cuts + blockIdx.x));
  const int c1 = __ldcg(&p.cuts[blockIdx.x].c1);
  const int n_tok = c4.x, tok0 = c4.y, head0 = c4.z, c0 = c4.w;
  if (n_tok == 0) return;
  const int G = p.group;
  const int inv_g = (65536 + G - 1) / G;   // r / G = r inv_g >> 16 for r < 128
  const int TT = p.decode ? p.toks_per_block : p.toks_per_block / kQTiles;   // tokens of a Q tile
  const int n_piece = c1 - c0 + 1;
  const uint32_t slot = uint32_t(p.item_rows) * kPartStride;
  for (int k = 0; k < kPairs; ++k) {
    const int rr = int(blockIdx.y) * kRows + 16 * k + row_in;
    const int r = rr % kBM, tok_t = (r * inv_g) >> 16, tok = rr / kBM * TT + tok_t;
    const bool live = r < TT * G && tok < n_tok;
    if (!__any_sync(0xffffffffu, live)) continue;
    const float* first = p.part + (size_t(2 * c0) + 1) * slot + uint32_t(rr) * kPartStride;
    const float* rest = first - slot;   // piece i > 0 lies 2 i slots on
    auto piece = [&](int i) { return i == 0 ? first : rest + size_t(2 * i) * slot; };
    constexpr int kStatOff = kHeadDim / 2;   // 32-bit word of m (then l) in a row
    float m = -INFINITY, l = 0.f;
    float acc[8] = {};
    for (int s0 = 0; s0 < n_piece; s0 += kBatch) {
      const float2 ml = (live && lane < kBatch && s0 + lane < n_piece)
                            ? __ldcg(reinterpret_cast<const float2*>(piece(s0 + lane) + kStatOff))
                            : make_float2(-INFINITY, 0.f);
      uint4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        v[j] = live && s0 + j < n_piece ? __ldcg(reinterpret_cast<const uint4*>(piece(s0 + j)) + lane)
                                        : make_uint4(0u, 0u, 0u, 0u);
      float mb = fmaxf(m, ml.x);
      for (int o = 8; o > 0; o >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
      const float mu = (mb == -INFINITY) ? 0.f : mb;
      if (s0 > 0) {
        const float sc = (m == -INFINITY) ? 0.f : ex2(m - mu);
        l *= sc;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] *= sc;
      }
      m = mb;
      const float wl = (ml.x == -INFINITY) ? ml.y : ml.y * ex2(ml.x - mu);   // l = 0 there, or nan
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float wgt = __shfl_sync(0xffffffffu, wl, j, 16);
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        l += wgt;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = f16x2_to_f32x2(w[i]);
          acc[2 * i] += x.x * wgt;
          acc[2 * i + 1] += x.y * wgt;
        }
      }
    }
    if (!live) continue;
    const float m_use = (m == -INFINITY) ? 0.f : m;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t orow = int64_t(tok0 + tok) * p.num_q_heads + head0 + (r - tok_t * G);
    uint4 out;
    out.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    out.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    out.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
    out.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
    reinterpret_cast<uint4*>(p.o + orow * kHeadDim)[lane] = out;
    if (lane == 0 && p.row_lse) p.row_lse[orow] = (m_use + __log2f(l)) * 0.69314718055994531f;
  }
}

// ---------------------------------------------------------------- launchers

cudaError_t launch_kv8_split_q(const Kv8Params& p, cudaStream_t stream) {
  const int64_t rows = int64_t(p.batch.total_q) * p.num_q_heads;
  return launch_pdl(kv8_split_q_kernel, dim3(unsigned((rows + 31) / 32)), dim3(256), 0, stream, 1, p, rows);
}

cudaError_t launch_kv8_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p,
                           int grid, cudaStream_t stream) {
  const size_t smem = f8::smem_bytes(p.batch.num_requests);
  static SmemAttr attr;
  cudaError_t e = ensure_smem_attr(kv8_fwd_kernel, attr, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_fwd_kernel, dim3(grid), dim3(f8::kThreads), smem, stream, 1, tq, tk, tv, p);
}

cudaError_t launch_kv8_combine(const Kv8Params& p, cudaStream_t stream) {
  if (p.split_tiles > 0)
    return launch_pdl(kv8_combine_kernel<8, 1, 4>, dim3(p.grid, p.item_rows / 16), dim3(256), 0, stream, 1, p);
  return launch_pdl(kv8_combine_kernel<4, 2, 6>, dim3(p.grid, (p.item_rows + 16) / 32), dim3(256), 0, stream, 1, p);
}

}  // namespace rag
