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
//       significands, so hi + lo is the value itself unless it lies 2^-14 or
//       more below the row's largest (then off by at most 2^-18 of that one)
//   S = hi K8 + lo K8: two kind::f8f6f4 products of twice the 16-bit rate, so
//       they cost what one bf16 product would, K tiles go from TMA to the
//       tensor core untouched, and no page is converted for the scores
//   score = S * (s_q * scale of the page): one factor per row and page, folded
//       into the softmax's multiply-add
// V enters as fp16 (code * scale, exact for scales that are powers of two):
// weights in e4m3 would lose what the softmax kept, and splitting them costs
// the issue-bound softmax warps more than two converting warps cost.
//   producer warp : per tile 8 + 8 TMA page boxes of 2 KB (K, V), the scales
//                   (loaded a tile ahead), the mask descriptor
//   MMA warp      : S_i = Q_i K8^T for both Q tiles, then O_i += P_i V
//   2 convert warps: V codes -> fp16 in the 128-byte swizzle, slots that hold
//                   no token zeroed
//   2 x 4 softmax warps: thread = row = TMEM lane; mask, online max and sum in
//                   the log2 domain, P (fp16) over the columns of S
// Every wait is bounded; a timeout raises a device error instead of hanging.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv8.cuh"
#include "params.cuh"

namespace rag {
namespace f8 {

constexpr int kKSt = 3;                          // K stages (codes)
constexpr int kRSt = 2;                          // V stages (codes)
constexpr int kVSt = 2;                          // V stages (fp16)
constexpr int kDescSlots = 4;
constexpr int kQTileBytes = 2 * kTile8;          // hi and lo
constexpr int kVTile = kBN * kHeadDim * 2;       // fp16
constexpr int kVHalf = kVTile / 2;               // 64 columns of d
constexpr int kThreads = 384;                    // 8 softmax + producer, MMA, 2 convert warps
constexpr float kRescale = 8.0f;                 // log2 units: rescale O when the max grows by > 2^8

// TMEM columns: S_i (P_i aliased over its first 64 columns), O_i
__host__ __device__ constexpr uint32_t col_s(int qt) { return 128u * qt; }
__host__ __device__ constexpr uint32_t col_o(int qt) { return 256u + 128u * qt; }

struct TileDesc {
  float ks[kPagesPerTile];
  int32_t lstart[kPagesPerTile];   // logical position of the page's slot 0
  uint8_t nvalid[kPagesPerTile];
  int32_t full;                    // every slot of the 8 pages is a token
  int32_t max_pos;                 // largest logical position of the tile
};
struct VInfo {
  float vs[kPagesPerTile];
  uint8_t nvalid[kPagesPerTile];
};

struct Ctrl {
  uint64_t q_full, q_empty;
  uint64_t kfull[kKSt], kempty[kKSt];
  uint64_t rfull[kRSt], rempty[kRSt];
  uint64_t vfull[kVSt], vempty[kVSt];
  uint64_t s_full[kQTiles], p_lo[kQTiles], p_hi[kQTiles], pv_done[kQTiles], o_full[kQTiles], o_free[kQTiles];
  uint64_t teardown;
  uint64_t desc_full[kDescSlots], desc_empty[kDescSlots];
  TileDesc desc[kDescSlots];
  VInfo vinfo[kRSt];
  ChunkCache chunks;
  Kv8Ring ring;
  uint32_t tmem_base;
  int32_t abort;
};

constexpr size_t kSmemData = size_t(kQTiles) * kQTileBytes + size_t(kKSt + kRSt) * kTile8 + size_t(kVSt) * kVTile;
constexpr size_t smem_bytes(int num_requests) {
  return 1024 + kSmemData + sizeof(Ctrl) + sizeof(int32_t) * (size_t(num_requests) + 1);
}
static_assert(smem_bytes(kMaxRequests) <= 227 * 1024, "shared memory of a CTA");

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

// K-major tile of 128 rows x 128 codes, 128B-swizzled; k-step kk covers codes [32 kk, 32 kk + 32).
__device__ __forceinline__ uint64_t code_desc(uint32_t base, int kk) { return sdesc_sw128(base + kk * 32, 16, 1024); }
// V tile [128 keys][128 d] fp16 as the B operand with N = d contiguous: k-step
// kk covers keys [16 kk, 16 kk + 16); the two 64-wide halves of d are 16 KB
// apart (leading byte offset), 8-key groups 1 KB apart (stride).
__device__ __forceinline__ uint64_t v_desc(uint32_t base, int kk) {
  return sdesc_sw128(base + kk * 16 * 128, kVHalf, 1024);
}

}  // namespace f8

using namespace f8;

__global__ void __launch_bounds__(f8::kThreads, 1)
kv8_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const Kv8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + kQTiles * kQTileBytes;
  uint8_t* sR = sK + kKSt * kTile8;
  uint8_t* sV = sR + kRSt * kTile8;
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
      mbar_init(&ctl->p_lo[q], 128);
      mbar_init(&ctl->p_hi[q], 128);
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
    uint32_t t_glob = 0;            // tiles seen by the CTA
    uint32_t n_sf0 = 0, n_sf1 = 0;  // completions of s_full[0] / s_full[1] consumed
    uint32_t n_pvq = 0;             // PVs into O_qt issued before the current step
    uint32_t n_of = 0;              // items whose O_qt has been read
    int bad = 0;
    pdl_wait();                     // the row scales come from the kernel before this one
    while (!bad && kv8_take<true>(&ctl->ring, n_it++, it, abort_flag, bad)) {
      const int n = it.n;
      // One Q tile: warpgroup 0 alone, alternating between the two S buffers
      // so that S of the next tile is computed during this tile's softmax.
      const int tok0 = it.rb * p.toks_per_block;
      const int n_qt = it.n_q - tok0 > TT ? 2 : 1;
      const bool single = n_qt == 1;
      const bool active = qt < n_qt;
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
        float cp[kPagesPerTile];
#pragma unroll
        for (int g = 0; g < kPagesPerTile; ++g) cp[g] = c_row * td->ks[g];
        // slots of each page that this row sees, a byte a page
        uint32_t nv_lo = 0x10101010u, nv_hi = 0x10101010u;
        const bool masked = !td->full || td->max_pos > lim;
        if (masked) {
          nv_lo = *reinterpret_cast<const uint32_t*>(&td->nvalid[0]);
          nv_hi = *reinterpret_cast<const uint32_t*>(&td->nvalid[4]);
          if (td->max_pos > lim) {
            uint32_t a = 0, b = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              a |= uint32_t(min(int((nv_lo >> (8 * g)) & 0xffu), max(lim - td->lstart[g] + 1, 0))) << (8 * g);
              b |= uint32_t(min(int((nv_hi >> (8 * g)) & 0xffu), max(lim - td->lstart[4 + g] + 1, 0))) << (8 * g);
            }
            nv_lo = a;
            nv_hi = b;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->desc_empty[slot]);
        if (!active) {
          // The other warpgroup uses S buffer 1 for the odd tiles; follow its
          // phases one by one. Descriptors run ahead of the products, and a
          // parity tells only neighbouring phases apart.
          if (i & 1) {
            if (!mbar_wait(&ctl->s_full[1], n_sf1 & 1, abort_flag)) { bad = 1; break; }
            ++n_sf1;
          }
          continue;
        }
        const int sb = single ? (i & 1) : qt;   // S buffer of this step
        const uint32_t s_addr = tmem + lane_off + col_s(sb);
        if (!mbar_wait(&ctl->s_full[sb], (sb ? n_sf1 : n_sf0) & 1, abort_flag)) { bad = 1; break; }
        tc_fence_after();
        if (!warp_live) {
          mbar_arrive(&ctl->p_lo[sb]);
          mbar_arrive(&ctl->p_hi[sb]);
          if (sb) ++n_sf1; else ++n_sf0;
          ++n_pvq;
          continue;
        }
        float x[kBN];
        {
          uint32_t u0[32], u1[32], u2[32], u3[32];
          tmem_ld32(s_addr + 0, u0);
          tmem_ld32(s_addr + 32, u1);
          tmem_ld32(s_addr + 64, u2);
          tmem_ld32(s_addr + 96, u3);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            x[j] = __uint_as_float(u0[j]);
            x[32 + j] = __uint_as_float(u1[j]);
            x[64 + j] = __uint_as_float(u2[j]);
            x[96 + j] = __uint_as_float(u3[j]);
          }
        }
        if (masked) {
#pragma unroll
          for (int c = 0; c < kBN; ++c) {
            const int pg = c >> 4;
            const uint32_t nv = ((pg < 4 ? nv_lo >> (8 * pg) : nv_hi >> (8 * (pg - 4))) & 0xffu);
            if (uint32_t(c & 15) >= nv) x[c] = -INFINITY;
          }
        }
        // row max: the largest raw score of each page, scaled by its factor (> 0)
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < kPagesPerTile; ++g) {
          const float* xg = x + 16 * g;
          float a = fmax3(xg[0], xg[1], xg[2]), b = fmax3(xg[3], xg[4], xg[5]);
          a = fmax3(a, xg[6], xg[7]);
          b = fmax3(b, xg[8], xg[9]);
          a = fmax3(a, xg[10], xg[11]);
          b = fmax3(b, xg[12], xg[13]);
          a = fmax3(a, xg[14], xg[15]);
          mx = fmaxf(mx, fmaxf(a, b) * cp[g]);
        }
        float alpha = 1.f;
        bool need = false;
        if (i == 0) {
          m_ref = mx;
        } else if (mx > m_ref + kRescale) {
          alpha = ex2(m_ref - mx);
          need = true;
        }
        if (__any_sync(0xffffffffu, need)) {
          // O must hold the previous tile's PV before it is rescaled. The PV
          // before that is complete (it was issued ahead of this tile's QK,
          // whose result is here), so the parity names exactly PV(n_pvq - 1).
          if (!mbar_wait(&ctl->pv_done[qt], (n_pvq - 1) & 1, abort_flag)) { bad = 1; break; }
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
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float c = cp[4 * h + (j >> 3)];
            const float2 y = ffma2(make_float2(x[64 * h + 2 * j], x[64 * h + 2 * j + 1]), make_float2(c, c), nm2);
            const float2 e = make_float2(ex2(y.x), ex2(y.y));
            ls[j & 3] = fadd2(ls[j & 3], e);
            pk[j] = pack_f16x2(e.x, e.y);
          }
          tmem_st32(s_addr + 32 * h, pk);   // P over the first 64 columns of S
          // publish this half of P: PV over its 64 keys may start
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(h == 0 ? &ctl->p_lo[sb] : &ctl->p_hi[sb]);
        }
        const float2 ls01 = fadd2(ls[0], ls[1]), ls23 = fadd2(ls[2], ls[3]);
        l_sum += (ls01.x + ls01.y) + (ls23.x + ls23.y);
        if (sb) ++n_sf1; else ++n_sf0;
        ++n_pvq;
      }
      if (bad) break;
      t_glob += n;
      // completions of s_full[1] that warpgroup 1 consumed in a two-Q-tile item
      // (all of them by the time O_0 is complete, which comes after the last)
      if (!single && qt == 0) n_sf1 += uint32_t(n);
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
      Kv8Walk walk;
      int cached_b = -1;
      kv8_line(p, prefix, &ctl->ring, lane);
      walk.start(&ctl->ring);
      while (!bad && walk.next(p, prefix, &ctl->ring, it)) {
        if (!kv8_put(&ctl->ring, n_it++, it, lane, abort_flag)) { bad = 1; break; }
        const int n = it.n;
        const int sub = lane & 7;
        auto page_id = [&](int tile) {
          return lane < 16 ? load_page_id(p.batch, walk.req, tile * kPagesPerTile + sub) : -1;
        };
        auto resolve = [&](int tile, int32_t id) {
          PageRef pg;
          pg.page = -1; pg.nvalid = 0; pg.lstart = 0; pg.chunk = -1;
          if (lane < 16)
            pg = page_ref_cached(&ctl->chunks, p.batch, walk.req, tile * kPagesPerTile + sub, id, p.num_pages,
                                 lane < 8 ? p.err : nullptr);
          return pg;
        };
        // page ids run two tiles ahead, scales one
        const int32_t first_id = page_id(it.t_begin);
        int32_t next_id = n > 1 ? page_id(it.t_begin + 1) : -1;
        if (walk.b != cached_b) {
          __syncwarp();
          load_chunk_cache(&ctl->chunks, p.batch, walk.req, lane);
          cached_b = walk.b;
        }
        PageRef pg = resolve(it.t_begin, first_id);
        float sc = page_scale_load(p, pg, it.g, lane);
        for (int i = 0; i < n; ++i) {
          const uint32_t t = t_glob + i;
          const int tile = it.t_begin + i;
          const PageRef cur = pg;
          const float scale = page_scale_ok(p, sc, lane);
          if (i + 1 < n) {
            pg = resolve(tile + 1, next_id);
            sc = page_scale_load(p, pg, it.g, lane);
            next_id = i + 2 < n ? page_id(tile + 2) : -1;
          }
          const uint32_t slot = t % kDescSlots;
          if (t >= kDescSlots && !mbar_wait(&ctl->desc_empty[slot], ((t / kDescSlots) - 1) & 1, abort_flag)) {
            bad = 1;
            break;
          }
          TileDesc* d = &ctl->desc[slot];
          const unsigned full_pages = __ballot_sync(0xffffffffu, lane < kPagesPerTile && cur.nvalid == kPage);
          const int last = lane < kPagesPerTile && cur.nvalid > 0 ? cur.lstart + cur.nvalid - 1 : -1;
          const int max_pos = __reduce_max_sync(0xffffffffu, last);
          if (lane < kPagesPerTile) {
            d->ks[lane] = scale;
            d->lstart[lane] = cur.lstart;
            d->nvalid[lane] = uint8_t(cur.nvalid);
          }
          if (lane == 0) { d->full = full_pages == 0xffu ? 1 : 0; d->max_pos = max_pos; }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->desc_full[slot]);
          const int box = cur.page >= 0 ? ((p.layer * p.num_pages + cur.page) * p.num_kv_heads + it.g) * kPage
                                        : -kPage;   // fully out of range: the box is zero-filled
          const int s = t % kKSt;
          if (t >= uint32_t(kKSt) && !mbar_wait(&ctl->kempty[s], ((t / kKSt) - 1) & 1, abort_flag)) { bad = 1; break; }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&ctl->kfull[s], kTile8);
          __syncwarp();
          if (lane < 8) tma_load_2d(sK + s * kTile8 + sub * kPageBytes8, &tm_k, &ctl->kfull[s], 0, box);
          ++n_k;
          const int sv = t % kRSt;
          if (t >= uint32_t(kRSt) && !mbar_wait(&ctl->rempty[sv], ((t / kRSt) - 1) & 1, abort_flag)) { bad = 1; break; }
          if (lane >= 8 && lane < 16) {
            ctl->vinfo[sv].vs[sub] = scale;
            ctl->vinfo[sv].nvalid[sub] = uint8_t(cur.nvalid);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&ctl->rfull[sv], kTile8);
          __syncwarp();
          if (lane >= 8 && lane < 16) tma_load_2d(sR + sv * kTile8 + sub * kPageBytes8, &tm_v, &ctl->rfull[sv], 0, box);
          ++n_v;
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
      // let every copy this warp issued land before the CTA exits
      if (lane == 0 && ctl->abort) {
        for (uint32_t t = n_k > kKSt ? n_k - kKSt : 0; t < n_k; ++t) wait_quiet(&ctl->kfull[t % kKSt], (t / kKSt) & 1);
        for (uint32_t t = n_v > kRSt ? n_v - kRSt : 0; t < n_v; ++t) wait_quiet(&ctl->rfull[t % kRSt], (t / kRSt) & 1);
      }
      __syncwarp();
    } else if (warp >= 10) {
      // ------------------------------------------------------------ convert warps
      // Warp 10 takes keys 0-63, warp 11 keys 64-127. A lane reads 16 codes of
      // a row and writes two 16-byte vectors of fp16; lanes of the upper half
      // of d write theirs in the other order, so that eight lanes cover all
      // banks with each store. Warp 10 also loads an item's Q tiles, which the
      // kernel before this one makes: the producer warp never waits for it, so
      // K and V stream in while the queries are still being split.
      const int base_row = (warp - 10) * 64;
      const int c = lane & 7;                         // 16 codes: columns 16c .. 16c + 15
      uint32_t t_glob = 0, q_iter = 0;
      int bad = 0;
      while (!bad && kv8_take<true>(&ctl->ring, n_it++, it, abort_flag, bad)) {
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
              tma_load_3d(sQ + q * kQTileBytes + kTile8, &tm_q, &ctl->q_full, kHeadDim, it.g * G,
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
          const uint8_t* src = sR + sr * kTile8;
          uint8_t* dst = sV + sv * kVTile + (c >> 2) * kVHalf;
#pragma unroll 4
          for (int j = 0; j < 16; ++j) {
            const int row = base_row + 4 * j + (lane >> 3);
            const int pgi = row >> 4;
            const bool live = (row & 15) < int(ctl->vinfo[sr].nvalid[pgi]);
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
      if (lane == 0 && q_iter > 0 && ctl->abort) wait_quiet(&ctl->q_full, (q_iter - 1) & 1);
      __syncwarp();
    } else {
      // ------------------------------------------------------------ MMA issuer (warp 9)
      if (lane == 0) {
        const uint32_t idesc_qk = idesc_e4m3_f32(kBM, kBN, 0, 0);
        const uint32_t idesc_pv = idesc_f16_f32(kBM, kHeadDim, 1);
        const uint32_t q_base = smem_u32(sQ);
        uint32_t t_glob = 0, q_iter = 0;
        uint32_t n_pf0 = 0, n_pf1 = 0;       // completions of p_lo/p_hi[0] and [1] consumed
        uint32_t n_item[kQTiles] = {0, 0};   // items begun, per Q tile
        int bad = 0;
        // S (buffer at column d) = (hi + lo) of the Q tile at qb times K codes at kb
        auto qk_mma = [&](uint32_t d, uint32_t qb, uint32_t kb) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_ss_f8(tmem + d, code_desc(qb, kk), code_desc(kb, kk), idesc_qk, kk > 0);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_f8(tmem + d, code_desc(qb + kTile8, kk), code_desc(kb, kk), idesc_qk, 1);
        };
        while (!bad && kv8_take<false>(&ctl->ring, n_it++, it, abort_flag, bad)) {
          const int n = it.n;
          const int n_qt = it.n_q - it.rb * p.toks_per_block > TT ? 2 : 1;
          if (!mbar_wait(&ctl->q_full, q_iter & 1, abort_flag)) { bad = 1; break; }
          tc_fence_after();
          if (n_qt == 1) {
            // One Q tile, two S buffers: QK of tiles 0 and 1 first, then per tile
            // i, PV(i) as soon as its P is written and QK(i + 2) into the buffer
            // PV(i) has just read (issue order keeps them apart).
            auto qk = [&](int j) {
              const uint32_t t = t_glob + j;
              const int s = t % kKSt;
              if (!mbar_wait(&ctl->kfull[s], (t / kKSt) & 1, abort_flag)) return false;
              tc_fence_after();
              qk_mma(col_s(j & 1), q_base, smem_u32(sK + s * kTile8));
              tc_commit(&ctl->s_full[j & 1]);
              tc_commit(&ctl->kempty[s]);
              if (j == n - 1) tc_commit(&ctl->q_empty);   // the rest of the item reads no Q
              return true;
            };
            for (int j = 0; j < n && j < 2 && !bad; ++j)
              if (!qk(j)) bad = 1;
            for (int i = 0; i < n && !bad; ++i) {
              const uint32_t t = t_glob + i;
              const int sv = t % kVSt;
              const int b = i & 1;
              if (!mbar_wait(&ctl->vfull[sv], (t / kVSt) & 1, abort_flag)) { bad = 1; break; }
              if (i == 0) {
                if (n_item[0] > 0 && !mbar_wait(&ctl->o_free[0], (n_item[0] - 1) & 1, abort_flag)) { bad = 1; break; }
                ++n_item[0];
              }
              uint32_t& npf = b ? n_pf1 : n_pf0;
              const uint32_t v_base = smem_u32(sV + sv * kVTile);
              bool ok = true;
              for (int hh = 0; hh < 2 && ok; ++hh) {
                if (!mbar_wait(hh == 0 ? &ctl->p_lo[b] : &ctl->p_hi[b], npf & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int kk = 4 * hh; kk < 4 * hh + 4; ++kk)
                  mma_ts(tmem + col_o(0), tmem + col_s(b) + kk * 8, v_desc(v_base, kk), idesc_pv, (i > 0) || (kk > 0));
              }
              if (!ok) { bad = 1; break; }
              ++npf;
              tc_commit(&ctl->pv_done[0]);
              if (i == n - 1) tc_commit(&ctl->o_full[0]);
              tc_commit(&ctl->vempty[sv]);
              if (i + 2 < n && !qk(i + 2)) { bad = 1; break; }
            }
            if (bad) break;
            t_glob += n;
            ++q_iter;
            continue;
          }
          // Tensor-core order per step: PV_0(t-1), QK_0(t), PV_1(t-1), QK_1(t), so
          // that softmax 0 of tile t runs while the pipe does PV_1 and QK_1.
          for (int i = 0; i <= n && !bad; ++i) {
            const uint32_t t = t_glob + i;          // tile of the QK products of this step
            const uint32_t tp = t - 1;              // tile of the PV products of this step
            const int s = t % kKSt;
            const int sv = tp % kVSt;
            uint32_t v_base = 0;
            const uint32_t k_base = smem_u32(sK + s * kTile8);
            if (i >= 1) {
              if (!mbar_wait(&ctl->vfull[sv], (tp / kVSt) & 1, abort_flag)) { bad = 1; break; }
              v_base = smem_u32(sV + sv * kVTile);
            }
            for (int q = 0; q < kQTiles && !bad; ++q) {
              if (i >= 1) {
                // O_q += P_q V for the previous tile
                if (i == 1) {
                  if (n_item[q] > 0 && !mbar_wait(&ctl->o_free[q], (n_item[q] - 1) & 1, abort_flag)) {
                    bad = 1;
                    break;
                  }
                  ++n_item[q];
                }
                uint32_t& npf = q ? n_pf1 : n_pf0;
                bool ok = true;
                for (int hh = 0; hh < 2 && ok; ++hh) {
                  if (!mbar_wait(hh == 0 ? &ctl->p_lo[q] : &ctl->p_hi[q], npf & 1, abort_flag)) { ok = false; break; }
                  tc_fence_after();
#pragma unroll
                  for (int kk = 4 * hh; kk < 4 * hh + 4; ++kk)
                    mma_ts(tmem + col_o(q), tmem + col_s(q) + kk * 8, v_desc(v_base, kk), idesc_pv,
                           (i > 1) || (kk > 0));
                }
                if (!ok) { bad = 1; break; }
                ++npf;
                tc_commit(&ctl->pv_done[q]);
                if (i == n) tc_commit(&ctl->o_full[q]);   // O_q of this item is complete
                if (q == kQTiles - 1) tc_commit(&ctl->vempty[sv]);   // the last read of this V stage
              }
              if (i < n) {
                // K of this tile is waited for only here, so that PV_0 of the
                // previous tile never waits on the next tile's load
                if (q == 0 && !mbar_wait(&ctl->kfull[s], (t / kKSt) & 1, abort_flag)) { bad = 1; break; }
                // S_q overwrites P_q (aliased over it), which PV_q of the previous
                // tile reads: tcgen05.mma operations of one CTA execute in issue
                // order, so no completion wait is needed.
                tc_fence_after();
                qk_mma(col_s(q), q_base + q * kQTileBytes, k_base);
                tc_commit(&ctl->s_full[q]);
              }
            }
            if (bad) break;
            if (i < n) tc_commit(&ctl->kempty[s]);
            // the drain step reads no Q: the next item's Q may load now
            if (i == n - 1) tc_commit(&ctl->q_empty);
          }
          if (bad) break;
          t_glob += n;
          ++q_iter;
        }
        if (bad) raise_abort(ctl, p.err);
        // every MMA issued so far completes before TMEM is released
        tc_commit(&ctl->teardown);
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
  float x[16];
  float amax = 0.f;
  bool odd = false;
  pdl_wait();   // q may be the previous kernel's output, and its attention may still read the split queries
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 u = src[k];
    const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * k + 2 * j] = __uint_as_float(uw[j] << 16);
      x[8 * k + 2 * j + 1] = __uint_as_float(uw[j] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float a = fabsf(x[j]);
    odd = odd || !(a < INFINITY);
    amax = fmaxf(amax, a);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const unsigned votes = __ballot_sync(0xffffffffu, odd);
  odd = (votes >> (threadIdx.x & 24)) & 0xffu;
  const int e = scale_exp(amax, kScaleExpMaxK);
  const float inv = pow2f(-e);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float y[4], d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = x[4 * k + j] * inv;
    hi[k] = e4m3x4(y[0], y[1], y[2], y[3]);
    const float2 h0 = f16x2_to_f32x2(e4m3x2_to_f16x2(hi[k] & 0xffffu));
    const float2 h1 = f16x2_to_f32x2(e4m3x2_to_f16x2(hi[k] >> 16));
    d[0] = y[0] - h0.x; d[1] = y[1] - h0.y; d[2] = y[2] - h1.x; d[3] = y[3] - h1.y;
    lo[k] = e4m3x4(d[0], d[1], d[2], d[3]);
  }
  if (row >= rows) return;
  uint8_t* dst = p.qs + row * (2 * kHeadDim) + 16 * c;
  *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(dst + kHeadDim) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  // inf and nan make the whole row nan, as in the product itself (inf - inf)
  if (c == 0) p.qscale[row] = odd ? __int_as_float(0x7fffffff) : pow2f(e);
}

// Merge the partial rows (O, m, l) of every cut unit:
//   m = max_s m_s, l = sum_s l_s 2^(m_s - m), O = sum_s O_s l_s 2^(m_s - m) / l.
// Block (c, y) merges rows 32 y .. 32 y + 31 of the unit whose second piece CTA
// c left (nothing for other CTAs); a warp takes a row at a time, each lane 4 of
// the 128 columns; lane j holds the statistics of piece s0 + j, and the O
// slices of kCombineBatch pieces are requested before any is used. (A warp per
// output row of the batch, each finding its own pieces, took 45 us on 16
// requests of 32-128 tokens.)
constexpr int kCombineBatch = 8;
constexpr int kCombineRows = 32;

__global__ void __launch_bounds__(256, 4) kv8_combine_kernel(const Kv8Params p) {
  pdl_launch_dependents();
  pdl_wait();   // partials and cuts come from the attention kernel
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 c4 = __ldcg(reinterpret_cast<const int4*>(p.cuts + blockIdx.x));
  const int c1 = __ldcg(&p.cuts[blockIdx.x].c1);
  const int n_tok = c4.x, tok0 = c4.y, head0 = c4.z, c0 = c4.w;
  if (n_tok == 0) return;
  const int G = p.group;
  const int TT = p.decode ? p.toks_per_block : p.toks_per_block / kQTiles;   // tokens of a Q tile
  const int n_piece = c1 - c0 + 1;
  const size_t slot = size_t(p.item_rows) * kPartStride;
  for (int rr = blockIdx.y * kCombineRows + warp; rr < min(p.item_rows, int(blockIdx.y + 1) * kCombineRows); rr += 8) {
    const int r = rr % kBM, tok = rr / kBM * TT + r / G;
    if (r >= TT * G || tok >= n_tok) continue;   // uniform over the warp
    const float* row0 = p.part + size_t(2 * c0) * slot + size_t(rr) * kPartStride;
    auto piece = [&](int i) { return row0 + (i == 0 ? slot : size_t(2 * i) * slot); };
    constexpr int kStatOff = kHeadDim / 2;   // 32-bit word of m (then l) in a row
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < n_piece; s0 += kCombineBatch) {
      const float2 ml = (lane < kCombineBatch && s0 + lane < n_piece)
                            ? __ldcg(reinterpret_cast<const float2*>(piece(s0 + lane) + kStatOff))
                            : make_float2(-INFINITY, 0.f);
      uint2 v[kCombineBatch];
#pragma unroll
      for (int j = 0; j < kCombineBatch; ++j)
        v[j] = s0 + j < n_piece ? __ldcg(reinterpret_cast<const uint2*>(piece(s0 + j)) + lane) : make_uint2(0u, 0u);
      float mb = fmaxf(m, ml.x);
      for (int o = 16; o > 0; o >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
      const float mu = (mb == -INFINITY) ? 0.f : mb;
      if (s0 > 0) {
        const float sc = (m == -INFINITY) ? 0.f : ex2(m - mu);
        l *= sc;
        acc.x *= sc; acc.y *= sc; acc.z *= sc; acc.w *= sc;
      }
      m = mb;
      const float wl = (ml.x == -INFINITY) ? ml.y : ml.y * ex2(ml.x - mu);   // l = 0 there, or nan
#pragma unroll
      for (int j = 0; j < kCombineBatch; ++j) {
        const float wgt = __shfl_sync(0xffffffffu, wl, j);
        const float2 lo = f16x2_to_f32x2(v[j].x), hi = f16x2_to_f32x2(v[j].y);
        l += wgt;
        acc.x += lo.x * wgt; acc.y += lo.y * wgt; acc.z += hi.x * wgt; acc.w += hi.y * wgt;
      }
    }
    const float m_use = (m == -INFINITY) ? 0.f : m;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t orow = int64_t(tok0 + tok) * p.num_q_heads + head0 + r % G;
    uint2 out;
    out.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    out.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(p.o + orow * kHeadDim)[lane] = out;
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
  return launch_pdl(kv8_combine_kernel, dim3(p.grid, (p.item_rows + kCombineRows - 1) / kCombineRows), dim3(256), 0,
                    stream, 1, p);
}

}  // namespace rag
