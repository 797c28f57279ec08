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
// An 8-bit append streams its rows through shared memory from this many page
// blocks of K an SM on, where the deeper read-ahead pays for a block's longer
// start, and from this many tokens a sequence on, as a sequence's unused units
// leave the long blocks unequal. Streamed / not, at 8 heads unless said: 4
// prompts of 256 tokens 9.5 / 7.4 us, of 512 (7 blocks an SM) 16.9 / 14.8, of
// 1,024 (14) 24.7 / 28.7, of 2,048 41.7 / 51.4; 16 of 700, 2 heads (9) 27.8 /
// 28.9; 2 of 2,048, 32 heads 38.9 / 53.0; 64 of 128 tokens 26.4 / 20.3, 32 of
// 192 15.4 / 16.9, 64 of 256 33.7 / 36.0.
constexpr int kStreamBlocksPerSm = 8;
constexpr int kStreamTokensPerSeq = 144;

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
  if (reinterpret_cast<uintptr_t>(device_err) & 3u) return RAG_ERR_INVALID_ARG;
  const int64_t n = seqs->total_new, out_bytes = n * q_row * elem;
  const auto span = [&](int64_t stride, int64_t row) { return ((n - 1) * stride + row) * elem; };
  if ((q != q_out && overlap(q_out, out_bytes, q, span(q_stride, q_row))) ||
      overlap(q_out, out_bytes, k, span(k_stride, kv_row)) || overlap(q_out, out_bytes, v, span(v_stride, kv_row)))
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
  // a power of two, as few as let every block (three an SM) start at once: its
  // table rows and index arithmetic serve all of a block's tokens. At 8 / 4 / 2
  // / 1 tokens a block, 16 prompts of up to 1,024 into 8 bits take 54 / 57 / 63
  // / 81 us and 5 prompts of up to 700 fp32 tokens 5.3 / 7.1 / 8.5 / 11.9.
  p.tokens_per_block = 1;
  while (p.tokens_per_block < 8 && seqs->total_new > 3 * p.tokens_per_block * num_sms()) p.tokens_per_block *= 2;
  p.kv_blocks = 0;
  return RAG_OK;
}

// ------------------------------------------------------------ attention

struct Kv8Plan {
  int decode;        // query blocks of at most 16 rows: the transposed kernel
  int split_tiles;   // key tiles of a piece, 0: equal stretches
  int cut;           // units may be cut: partial rows and a combine
  int grid, toks_per_block, item_rows;
};

// Units of at most this many key tiles are not cut: one CTA walks them in less
// time than the combine's launch and its reads of partial rows take (a step
// over 5 tiles: 8.8 us cut in pieces of two, 9.7 us whole).
constexpr int kWholeTiles = 2;
// A piece's start and end (first loads, last products, its rows), in tiles.
// (Counted as 8, the step of 16 requests is cut into pieces: 47 us against 38;
// 2 gives the same plans as 4.)
constexpr double kPieceTiles = 4.0;

// The kernel is one choice a batch, by its longest query block: both kernels on
// one line of work would need a line each. A batch that mixes the kinds is faster
// as two calls: 63 single tokens over about 12,900 keys and a prompt of 100 over
// 10,000 take 651 us in one, 329 in two; 15 over 3,900 and 100 over 4,000 84 and
// 73; 63 over 1,000 and 40 over 1,000 90 and 64; 7 and a prompt of 400 over 10,000
// each 150 and 140.
static Kv8Plan plan_kv8(const rag_batch& b, int num_kv_heads, int group, int sms) {
  Kv8Plan pl;
  pl.decode = int64_t(b.max_q) * group <= 16 ? 1 : 0;
  pl.toks_per_block = pl.decode ? std::max(1, 16 / group) : kQTiles * (kBM / group);   // any group, if no request has queries
  pl.item_rows = pl.decode ? 16 : kFwdRows;
  // two CTAs of the decode kernel share an SM; no more CTAs than the batch's
  // capacities can give work to
  const int pages = kv8_tile_pages(pl.decode);
  const int tiles_max = std::max(1, cdiv(b.max_pages, pages));
  pl.cut = tiles_max > kWholeTiles ? 1 : 0;
  const double rt = cdiv(b.max_q, pl.toks_per_block);
  const double most = !pl.cut ? double(num_kv_heads) * (cdiv(b.total_q, pl.toks_per_block) + b.num_requests)
                              : num_kv_heads * rt * (double(b.num_page_refs) / pages + 2.0 * b.num_requests) *
                                    (pl.decode ? 1 : kCost2) / (pl.decode ? kMinWorkDecode : kMinWork);
  pl.grid = int(std::max(1.0, std::min(double(pl.decode ? 2 * sms : sms), most)));
  pl.split_tiles = tiles_max;
  if (pl.cut) {
    // One piece a CTA, or equal stretches with up to two pieces' starts and
    // ends in a CTA. Requests of unlike lengths round up to half a piece a
    // unit more; if that is not enough on the device, it uses stretches.
    const double B = std::max(1, b.num_requests);
    const double units = num_kv_heads * B * std::max(1, cdiv(cdiv(b.total_q, int(B)), pl.toks_per_block));
    const double tiles = B == 1 ? tiles_max : double(b.num_page_refs) / pages / B + 0.5;
    const double room = B == 1 ? std::floor(pl.grid / units) : pl.grid / units - 0.5;
    const double ts = room >= 1.0 ? std::ceil(tiles / room) : 0.0;
    pl.split_tiles = ts > 0.0 && ts + kPieceTiles <= units * tiles / pl.grid + 2 * kPieceTiles ? std::max(2, int(ts)) : 0;
  }
  return pl;
}

// Workspace (bytes, each region 256-aligned): error word, split queries, their
// row scales, the cuts, two partial slots per CTA (when units are cut).
struct Kv8Ws {
  size_t off_qs, off_qscale, off_cuts, off_part, total;
};
static Kv8Ws ws_kv8(const rag_batch& b, int num_q_heads, const Kv8Plan& pl) {
  Kv8Ws w;
  const size_t rows = pl.decode ? 0 : size_t(b.total_q) * num_q_heads;   // the decode kernel splits its own queries
  size_t at = 256;
  w.off_qs = at; at = align256(at + rows * 2 * kHeadDim);
  w.off_qscale = at; at = align256(at + rows * sizeof(float));
  w.off_cuts = at; at = align256(at + (pl.cut ? size_t(pl.grid) * sizeof(Kv8Cut) : 0));
  w.off_part = at;
  if (pl.cut) at = align256(at + size_t(2) * pl.grid * pl.item_rows * kPartStride * sizeof(float));
  w.total = at;
  return w;
}

static rag_status check_kv8_attn(const rag_kv8_pool* pool, const rag_batch* batch, int32_t num_q_heads) {
  rag_status st = check_pool8(pool);
  if (st != RAG_OK) return st;
  st = check_batch(batch);
  if (st != RAG_OK) return st;
  if (num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0) return RAG_ERR_SHAPE;
  const int G = num_q_heads / pool->num_kv_heads;
  if (G > kBM) return RAG_ERR_UNSUPPORTED;
  // the units' weights are counted in 31 bits
  const rag_batch& b = *batch;
  const Kv8Plan pl = plan_kv8(b, pool->num_kv_heads, G, 1);
  const double tiles = double(b.num_page_refs) / kv8_tile_pages(pl.decode) + 2.0 * b.num_requests;
  if (tiles * pool->num_kv_heads * (double(cdiv(b.max_q, pl.toks_per_block)) + 1) * kCost2 >= 2147483648.0) return RAG_ERR_UNSUPPORTED;
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
  const int64_t units = int64_t(seqs->total_new) / kPage + 2 * int64_t(seqs->n_seqs);   // see kv8_append_kernel
  const int q_blocks = q ? cdiv(seqs->total_new, p.tokens_per_block) : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (int64_t(seqs->total_new) / kPage * p.num_kv_heads >= kStreamBlocksPerSm * int64_t(num_sms()) &&
      seqs->total_new >= kStreamTokensPerSeq * int64_t(seqs->n_seqs)) {
    // many tokens: rows streamed through shared memory, queries in a launch of their own
    const int slots = 2 * num_sms();
    int64_t best = INT64_MAX;
    for (int n = 1; n <= 8; ++n) {   // units a block: the fewest rounds of blocks, then the longest blocks
      const int64_t rounds = cdiv(cdiv(units, n), slots) * int64_t(n);
      if (rounds <= best) {
        best = rounds;
        p.units_per_block = n;
      }
    }
    // fewer units than blocks the GPU holds: a unit's stages over several
    // blocks (2 prompts of 512 tokens, 32 heads: 22.7 us -> 13.4). Never for
    // its balance alone: two blocks a unit slow 32 chunks of 2,048 tokens from
    // 99 to 145 us.
    const int groups = cdiv(2 * p.num_kv_heads, 8);
    p.heads_split = int(std::max<int64_t>(1, std::min<int64_t>(groups, slots / units)));
    {
      LaunchScope ls(kKindKv8Append, s);
      cudaError_t e = launch_kv8_append_stream(p, cdiv(units, p.units_per_block) * p.heads_split, s);
      ls.done(e);
      if (e != cudaSuccess) return RAG_ERR_CUDA;
    }
    if (q) {
      LaunchScope ls(kKindRopeQ, s);
      cudaError_t e = launch_rope_q(p, q_blocks, s);
      ls.done(e);
      if (e != cudaSuccess) return RAG_ERR_CUDA;
    }
    return RAG_OK;
  }
  // a block takes several units once the GPU is filled a few times over: its
  // start (sequence, page ids) is paid once for them. With 1 / 2 / 4 / 8 at most,
  // 32 query heads with 8 KV heads: 512 sequences of 64 tokens 185 / 179 / 179 /
  // 179 us (two is the rule's choice), 1,024 of 64 365 / 351 / 343 / 342 (five),
  // 4,096 of 1 119 / 99 / 87 / 81 (seven); K and V alone: 4,096 of 16, 8 heads
  // 215 / 189 / 174 / 174 (eight), 4,096 of 32, 1 head 219 / 190 / 156 / 144. With
  // fewer units than SMs a block takes 8 page blocks of one, so that no warp takes two
  // (64 tokens of 64 sequences 4.9 us against 5.8, 4 prompts of 256 7.5 against
  // 8.3; but 64 prompts of 16 tokens, 192 units, 9.8 against 8.9)
  p.units_per_block = int(std::max<int64_t>(1, std::min<int64_t>(8, units / (8 * num_sms()))));
  p.heads_split = units < num_sms() ? cdiv(2 * p.num_kv_heads, 8) : 1;
  const int64_t kv_blocks = (units + p.units_per_block - 1) / p.units_per_block * p.heads_split;
  if (kv_blocks + q_blocks >= (int64_t(1) << 31)) return RAG_ERR_UNSUPPORTED;
  p.kv_blocks = int(kv_blocks);
  LaunchScope ls(kKindKv8Append, s);
  cudaError_t e = launch_kv8_append(p, int(kv_blocks + q_blocks), s);
  ls.done(e);
  return e == cudaSuccess ? RAG_OK : RAG_ERR_CUDA;
}

size_t rag_kv8_workspace_size(const rag_kv8_pool* pool, const rag_batch* batch, int32_t num_q_heads) {
  if (check_kv8_attn(pool, batch, num_q_heads) != RAG_OK) return 0;
  return ws_kv8(*batch, num_q_heads, plan_kv8(*batch, pool->num_kv_heads, num_q_heads / pool->num_kv_heads, num_sms())).total;
}

rag_status rag_kv8_attn(const rag_kv8_pool* pool, int32_t layer, const rag_batch* batch, const void* q,
                        int32_t num_q_heads, float sm_scale, int32_t causal, void* o, float* row_lse, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const rag_status st = check_kv8_attn(pool, batch, num_q_heads);
  if (st != RAG_OK) return st;
  if (layer < 0 || layer >= pool->num_layers) return RAG_ERR_INVALID_ARG;
  const rag_batch& b = *batch;
  if (b.total_q > 0 && (!q || !o)) return RAG_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || (reinterpret_cast<uintptr_t>(row_lse) & 3u)) return RAG_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale)) return RAG_ERR_INVALID_ARG;
  const int64_t q_bytes = int64_t(b.total_q) * num_q_heads * kHeadDim * 2;
  if (overlap(q, q_bytes, o, q_bytes)) return RAG_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return RAG_ERR_WORKSPACE;
  const int H = pool->num_kv_heads, G = num_q_heads / H;
  const Kv8Plan pl = plan_kv8(b, H, G, num_sms());
  const Kv8Ws ws = ws_kv8(b, num_q_heads, pl);
  if (workspace_bytes < ws.total) return RAG_ERR_WORKSPACE;
  if (b.num_requests == 0 || b.total_q == 0) return RAG_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  Kv8Params p = {};
  p.batch = to_dev(b);
  p.num_pages = pool->num_pages;
  p.num_kv_heads = H;
  p.num_q_heads = num_q_heads;
  p.group = G;
  p.layer = layer;
  p.toks_per_block = pl.toks_per_block;
  p.item_rows = pl.item_rows;
  p.decode = pl.decode;
  p.split_tiles = pl.split_tiles;
  p.grid = pl.grid;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = (sm_scale > 0.f ? std::max(sm_scale, kSmScaleMin) : 1.0f / std::sqrt(float(kHeadDim))) * 1.4426950408889634f;
  p.k_scale = pool->k_scale;
  p.v_scale = pool->v_scale;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.qs = base + ws.off_qs;
  p.qscale = reinterpret_cast<float*>(base + ws.off_qscale);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.row_lse = row_lse;
  p.part = pl.cut ? reinterpret_cast<float*>(base + ws.off_part) : nullptr;
  p.cuts = reinterpret_cast<Kv8Cut*>(base + ws.off_cuts);
  p.err = reinterpret_cast<int32_t*>(base);

  CUtensorMap tm_q, tm_k, tm_v;
  {
    const uint64_t dp[2] = {uint64_t(kHeadDim), uint64_t(pool->num_layers) * pool->num_pages * H * kPage};
    const uint64_t sp[1] = {uint64_t(kHeadDim)};
    const uint32_t bp[2] = {uint32_t(kHeadDim), uint32_t(kPage)};
    if (!make_map(&tm_k, pool->k, 2, dp, sp, bp, true) || !make_map(&tm_v, pool->v, 2, dp, sp, bp, true))
      return RAG_ERR_CUDA;
  }
  if (pl.decode) {
    LaunchScope ls(kKindKv8Decode, s);
    cudaError_t e = launch_kv8_decode(tm_k, tm_v, p, pl.grid, s);
    ls.done(e);
    if (e != cudaSuccess) return RAG_ERR_CUDA;
  } else {
    const uint64_t dq[3] = {2u * kHeadDim, uint64_t(num_q_heads), uint64_t(b.total_q)};
    const uint64_t sq[2] = {2u * kHeadDim, uint64_t(num_q_heads) * 2 * kHeadDim};
    const uint32_t bq[3] = {uint32_t(kHeadDim), uint32_t(G), uint32_t(kBM / G)};
    if (!make_map(&tm_q, p.qs, 3, dq, sq, bq, true)) return RAG_ERR_CUDA;
    {
      LaunchScope ls(kKindKv8SplitQ, s);
      cudaError_t e = launch_kv8_split_q(p, s);
      ls.done(e);
      if (e != cudaSuccess) return RAG_ERR_CUDA;
    }
    LaunchScope ls(kKindKv8Attn, s);
    cudaError_t e = launch_kv8_fwd(tm_q, tm_k, tm_v, p, pl.grid, s);
    ls.done(e);
    if (e != cudaSuccess) return RAG_ERR_CUDA;
  }
  if (pl.cut) {
    LaunchScope ls(kKindKv8Combine, s);
    cudaError_t e = launch_kv8_combine(p, s);
    ls.done(e);
    if (e != cudaSuccess) return RAG_ERR_CUDA;
  }
  return RAG_OK;
}

}  // extern "C"
