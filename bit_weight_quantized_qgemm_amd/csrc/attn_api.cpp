// C-ABI front end of the attention operators: argument validation (before any
// HIP call), the split of the cache's length and kernel dispatch. See
// include/qgemm.h for the contract.
#include "qgemm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_internal.h"

namespace {

constexpr int64_t kMaxSeqs = 65535;
constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxLen = int64_t(1) << 24;
constexpr int kMaxKvHeads = 1024;
constexpr int kMaxGroup = 128;
constexpr int64_t kMaxTokenStride = int64_t(1) << 25;

std::atomic<int> g_force_splits{0};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_act(int dt) { return dt == QGEMM_DT_F16 || dt == QGEMM_DT_BF16; }

bool positive(float x) { return std::isfinite(x) && x > 0.f; }

// A tensor's bytes in memory: [first, last).
struct Extent {
  uintptr_t first = 0, last = 0;
};

bool overlap(const Extent& a, const Extent& b) { return a.first < b.last && b.first < a.last; }

Extent extent(const void* p, int64_t elems, int64_t elt) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return p && elems > 0 ? Extent{a, a + (uintptr_t)(elems * elt)} : Extent{};
}

// [tokens][heads][dim] with the given strides
Extent extent3(const void* p, int64_t tokens, int64_t ts, int64_t heads, int64_t hs, int64_t dim) {
  return extent(p, (tokens - 1) * ts + (heads - 1) * hs + dim, 2);
}

// A stride that n places are apart by: not used where there is one.
bool valid_step(int64_t n, int64_t stride, int64_t multiple, int64_t most) {
  return n == 1 || (stride >= 0 && stride <= most && stride % multiple == 0);
}
// Strides of a [tokens][heads][dim] tensor: 16-byte rows that do not overlap
// within a token; bounded so that no extent overflows.
bool valid_strides(int64_t tokens, int64_t ts, int64_t heads, int64_t hs, int64_t dim) {
  constexpr int64_t kMost = int64_t(1) << 32;
  return valid_step(tokens, ts, 8, kMost) && valid_step(heads, hs, 8, kMost) && (heads == 1 || hs >= dim);
}
// ... of one that is written: its tokens must not overlap either.
bool valid_out_strides(int64_t tokens, int64_t ts, int64_t heads, int64_t hs, int64_t dim) {
  return valid_strides(tokens, ts, heads, hs, dim) &&
         (tokens == 1 || ts >= (heads - 1) * hs + dim || (ts >= dim && hs >= (tokens - 1) * ts + dim));
}

int check_cache(const qgemm_kv_cache* c, int act_dtype) {
  if (c->kv_heads < 1 || c->kv_heads > kMaxKvHeads) return QGEMM_ERR_SHAPE;
  if (c->head_dim < 16 || c->head_dim > qg::kMaxHeadDim || c->head_dim % 16 != 0) return QGEMM_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16 != 0) return QGEMM_ERR_SHAPE;
  if (c->num_pages < 1 || c->num_pages > INT32_MAX) return QGEMM_ERR_SHAPE;
  if (c->dtype != QGEMM_DT_F16 && c->dtype != QGEMM_DT_BF16 && c->dtype != QGEMM_DT_FP8) return QGEMM_ERR_RANGE;
  if (c->dtype != QGEMM_DT_FP8 && c->dtype != act_dtype) return QGEMM_ERR_RANGE;
  if (!positive(c->k_scale) || !positive(c->v_scale)) return QGEMM_ERR_RANGE;
  if (c->dtype != QGEMM_DT_FP8 && (c->k_scale != 1.f || c->v_scale != 1.f)) return QGEMM_ERR_RANGE;
  if (!c->k || !c->v) return QGEMM_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return QGEMM_ERR_ALIGN;
  const int64_t step = c->dtype == QGEMM_DT_FP8 ? 16 : 8;
  constexpr int64_t kMost = int64_t(1) << 40;
  if (c->token_stride < c->head_dim || c->token_stride > kMaxTokenStride || c->token_stride % step != 0)
    return QGEMM_ERR_ALIGN;
  if (!valid_step(c->kv_heads, c->head_stride, step, kMost) || (c->kv_heads > 1 && c->head_stride < c->head_dim))
    return QGEMM_ERR_ALIGN;
  // 2^31 pages of 2^30 elements stay below 2^62
  if (!valid_step(c->num_pages, c->page_stride, step, int64_t(1) << 30)) return QGEMM_ERR_ALIGN;
  return QGEMM_OK;
}

Extent cache_extent(const qgemm_kv_cache* c, const void* p) {
  const int64_t elems = (c->num_pages - 1) * c->page_stride + (c->page_size - 1) * c->token_stride +
                        (c->kv_heads - 1) * c->head_stride + c->head_dim;
  return extent(p, elems, c->dtype == QGEMM_DT_FP8 ? 1 : 2);
}

qg::CacheArgs cache_args(const qgemm_kv_cache* c, const int32_t* table, int64_t table_stride) {
  qg::CacheArgs a{};
  a.k = c->k;
  a.v = c->v;
  a.page_stride = c->page_stride;
  a.token_stride = c->token_stride;
  a.head_stride = c->head_stride;
  a.table = table;
  a.table_stride = table_stride;
  a.num_pages = (int32_t)c->num_pages;
  a.page_blocks = c->page_size / qg::kTokBlock;
  const uint64_t d = (uint64_t)a.page_blocks;
  a.magic = d == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + d - 1) / d);
  return a;
}

int check_heads(int32_t q_heads, int32_t kv_heads) {
  if (q_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > kMaxGroup) return QGEMM_ERR_SHAPE;
  return QGEMM_OK;
}

// What the callers' window and sinks mean for contexts of up to max_len tokens: a
// window beyond every position is none (0, and then there are no sinks), sinks beyond
// the context are all of it. Plans and kernels take these alone, so that both see the
// same tokens and sums over them stay small whatever the caller passed.
struct Mask {
  int64_t window, sinks;
};
Mask bounded_mask(int64_t max_len, int64_t window, int64_t sinks) {
  if (window >= max_len) return Mask{0, 0};
  return Mask{window, window == 0 ? 0 : std::min(sinks, max_len)};
}

// Most token blocks that a sequence has to visit.
int64_t visible_blocks(int64_t max_len, int64_t rows, const Mask& mask) {
  const int64_t all = (max_len + qg::kTokBlock - 1) / qg::kTokBlock;
  if (mask.window == 0) return all;
  return std::min(all, (mask.sinks + qg::kTokBlock - 1) / qg::kTokBlock +
                           (mask.window + rows - 1 + 2 * qg::kTokBlock - 2) / qg::kTokBlock);
}

void split(qg::AttnPlan& pl, int64_t blocks, int64_t want, int step, int head_dim) {
  const int force = g_force_splits.load();
  int64_t splits = force ? force : std::max<int64_t>(1, want);
  // more tiles than the workspace has counters fill the device without a split
  if (pl.tiles > qg::kMaxCounters) splits = 1;
  blocks = std::max<int64_t>(1, blocks);
  const int64_t per = (blocks + splits - 1) / splits;
  pl.split_blocks = (int)((per + step - 1) / step * step);
  pl.splits = (int)((blocks + pl.split_blocks - 1) / pl.split_blocks);
  pl.ws_bytes = 0;
  if (pl.splits > 1) {
    const size_t parts = (size_t)pl.tiles * pl.splits;
    pl.stats_offset = qg::kCounterBytes;
    pl.partial_offset = pl.stats_offset + qg::align256(parts * pl.part_rows * 8);
    pl.ws_bytes = pl.partial_offset + parts * pl.part_rows * head_dim * 4;
  }
}

qg::AttnPlan decode_plan(int64_t num_seqs, int64_t max_len, int q_heads, int kv_heads, int head_dim,
                         const Mask& mask) {
  qg::AttnPlan pl;
  const int group = q_heads / kv_heads;
  pl.row_tiles = (group + qg::kDecodeRows - 1) / qg::kDecodeRows;
  pl.part_rows = std::min(group, qg::kDecodeRows);
  pl.tiles = num_seqs * kv_heads * pl.row_tiles;
  const int64_t blocks = visible_blocks(max_len, 1, mask);
  constexpr int kStep = 2 * qg::kDecodeWaves;   // one pair of blocks for each wave
  const int64_t steps = (blocks + kStep - 1) / kStep;
  // Parts of a tile, by tiles per compute unit and steps (128 tokens) of the longest
  // context. Joining costs about 3 us, a step of a lone workgroup 1.6. Measured on 8
  // key-value heads of 128, 16 bits, us (one length / ragged up to it):
  //  - up to 3 steps: unsplit (12 x 256 tokens 7.8, in two parts 9.2).
  //  - up to a tile per four units: one part per unit, which streams as fast as more
  //    and joins fewer (8 x 4096 in 4 parts 26 / 23, in 8 27 / 24); beyond 16 parts,
  //    which the join reads in one go, only while each keeps four steps (4 x 8192, one
  //    head: 15 in 16 parts, 21 in 64). Heads above 128 values leave room for one
  //    workgroup per unit: the same up to any number of tiles (16 x 4000, 8 heads of
  //    256: 85 in 2 parts, 101 in 8).
  //  - up to a tile per two units: four parts per unit, whose order of starting evens
  //    out contexts of different lengths (16 x 4096 in 8 parts 49 / 32, in 2 45 / 36);
  //    two parts below 16 steps (16 x 1024 in 2 17 / 15, in 8 20 / 17).
  //  - up to two tiles per unit: four parts at least, once each keeps eight steps (32
  //    x 4096 in 4 parts 87 / 58, unsplit 80 / 64; 63 x 8192 321 / 182 and 301 / 225;
  //    but 32 x 2048 49 / 33 and 42 / 34, 32 x 512 21 / 17 and 14 / 12); three steps
  //    where whole tiles would leave a fifth of the units idle (40 x 1500 in 4 parts
  //    48 / 39, unsplit 53 / 39; 40 x 3000 84 / 59 and 100 / 77).
  //  - beyond, the tiles themselves fill the device (96 x 4096 unsplit 233 / 165, in
  //    two parts 248 / 170).
  const int64_t cus = qg::device_cu_count(), tiles = pl.tiles;
  int64_t parts = 1;
  if (steps > 3 && tiles < 2 * cus) {
    const bool even = (tiles + cus - 1) / cus * cus * 4 <= 5 * tiles;
    if (tiles <= cus / 4 || head_dim > 128) parts = std::min({cus / tiles, steps, std::max<int64_t>(16, steps / 4)});
    else if (tiles <= cus / 2) parts = steps < 16 ? 2 : std::min(4 * cus / tiles, steps / 2);
    else if (steps >= (even ? 32 : 12)) parts = std::max<int64_t>(4, 4 * cus / tiles);
  }
  split(pl, blocks, parts, kStep, head_dim);
  return pl;
}

qg::AttnPlan prefill_plan(int64_t num_seqs, int64_t max_q, int64_t max_len, int q_heads, int kv_heads, int head_dim,
                          const Mask& mask) {
  qg::AttnPlan pl;
  const int64_t rows = max_q * (q_heads / kv_heads);
  pl.row_tiles = (int)((rows + qg::kPrefillRows - 1) / qg::kPrefillRows);
  pl.part_rows = (int)std::min<int64_t>(rows, qg::kPrefillRows);
  pl.tiles = num_seqs * kv_heads * pl.row_tiles;
  const int64_t blocks = visible_blocks(max_len, std::min<int64_t>(max_q, qg::kPrefillRows), mask);
  // Tiles of K and V hold 64 tokens (32 for heads above 128 values). One takes a
  // workgroup that has a compute unit for itself 1.25 us, and w of them that share a
  // unit 1.15 w us together (0.9 and 0.65 w for heads of 64); a join of s parts, x MB,
  // costs 2 + 0.08 s + 2.8 sqrt(x) us (16 parts are read at a time), with 0.45 x beyond
  // 40 MB, where the parts leave the caches. A split has to win 5 %. Of 197 shapes
  // (1..512 new tokens on 600..200000, 64 to 256 values, 1..16 sequences) the split
  // that this finds is on average 2 % slower than the best of 1..256 parts (50 tokens
  // on 20000, 64/8 heads: 58 us, best 54, unsplit 329; 12 x 40 on 12000, 32/8 heads of
  // 64, e4m3: 99, best 95, unsplit 174). Where a good part of the context is new, the
  // row tiles see less of it the earlier they stand, and fill the units in whatever
  // order they end: then the mean work counts, and the longest tile (4096 new tokens,
  // 20/20 heads of 80, 640 row tiles: 95 us, in two parts 122).
  const int kStep = head_dim <= 128 ? 4 : 2;   // blocks of a tile of K and V
  const int cus = qg::device_cu_count();
  int best = 1;
  if (pl.tiles <= 4 * cus) {
    const int steps = (int)((blocks + kStep - 1) / kStep), tiles = (int)pl.tiles;
    const double part_mb = (double)tiles * pl.part_rows * head_dim * 4e-6;
    const double alone = head_dim <= 64 ? 0.9 : 1.25, shared = head_dim <= 64 ? 0.65 : 1.15;
    const bool even = mask.window != 0 || max_q * 5 < max_len;
    const double mean = even ? 1 : 1 - 0.5 * std::min(max_q, max_len) / (double)max_len;   // of a tile's visible part
    double least = 0;
    for (int s = 1; s <= steps && s * tiles <= 8 * cus && s <= 2 * cus; s += s < 32 ? 1 : 16) {
      const int turns = (steps + s - 1) / s, on_unit = (tiles * s + cus - 1) / cus;
      const double mb = part_mb * s, join = s == 1 ? 0 : 2 + 0.08 * s + std::max(2.8 * std::sqrt(mb), 0.45 * mb);
      const double work = even ? shared * on_unit : shared * mean * tiles * s / cus;
      const double cost = turns * (on_unit == 1 ? alone : std::max(alone, work)) + join;
      if (s == 1 || cost < least * (best == 1 ? 0.95 : 1)) {
        least = cost;
        best = s;
      }
    }
  }
  split(pl, blocks, best, kStep, head_dim);
  return pl;
}

int check_attn_shape(int64_t num_seqs, int64_t max_len, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                     int64_t window, int32_t sinks) {
  if (num_seqs < 0 || num_seqs > kMaxSeqs) return QGEMM_ERR_SHAPE;
  if (max_len < 0 || max_len > kMaxLen) return QGEMM_ERR_SHAPE;
  if (kv_heads < 1 || kv_heads > kMaxKvHeads) return QGEMM_ERR_SHAPE;
  if (head_dim < 16 || head_dim > qg::kMaxHeadDim || head_dim % 16 != 0) return QGEMM_ERR_SHAPE;
  if (window < 0 || sinks < 0) return QGEMM_ERR_RANGE;
  return check_heads(q_heads, kv_heads);
}

int run_attn(const qgemm_attn_call& g, bool prefill) {
  const qgemm_kv_cache* c = g.cache;
  const int64_t num_tokens = prefill ? g.num_tokens : g.num_seqs, max_q = prefill ? g.max_q : 1;
  const int32_t* q_start = prefill ? g.q_start : nullptr;
  if (!c) return QGEMM_ERR_NULL;
  if (!valid_act(g.act_dtype)) return QGEMM_ERR_RANGE;
  int st = check_attn_shape(g.num_seqs, g.max_len, g.q_heads, c->kv_heads, c->head_dim, g.window, g.sinks);
  if (st) return st;
  if (num_tokens < 0 || num_tokens > kMaxTokens || max_q < 0 || max_q > kMaxTokens) return QGEMM_ERR_SHAPE;
  st = check_cache(c, g.act_dtype);
  if (st) return st;
  if (!positive(g.scale) || !positive(g.scale * c->k_scale)) return QGEMM_ERR_RANGE;
  if (g.num_seqs == 0 || num_tokens == 0 || max_q == 0) return QGEMM_OK;
  if (!g.q || !g.out || !g.seq_lens || (!g.block_table && g.table_stride > 0) || (prefill && !q_start))
    return QGEMM_ERR_NULL;
  if (!aligned(g.q, 16) || !aligned(g.out, 16) || !aligned(g.seq_lens, 4) || !aligned(g.block_table, 4) ||
      !aligned(q_start, 4))
    return QGEMM_ERR_ALIGN;
  if (!valid_strides(num_tokens, g.q_token_stride, g.q_heads, g.q_head_stride, c->head_dim) ||
      !valid_out_strides(num_tokens, g.out_token_stride, g.q_heads, g.out_head_stride, c->head_dim))
    return QGEMM_ERR_ALIGN;
  if (g.table_stride < 0 || g.table_stride > kMaxLen || g.max_len > g.table_stride * c->page_size)
    return QGEMM_ERR_SHAPE;

  const Mask mask = bounded_mask(g.max_len, g.window, g.sinks);
  const qg::AttnPlan pl = prefill
                              ? prefill_plan(g.num_seqs, max_q, g.max_len, g.q_heads, c->kv_heads, c->head_dim, mask)
                              : decode_plan(g.num_seqs, g.max_len, g.q_heads, c->kv_heads, c->head_dim, mask);
  if (pl.tiles * pl.splits > INT32_MAX) return QGEMM_ERR_SHAPE;
  if (pl.ws_bytes > 0) {
    if (!g.workspace) return QGEMM_ERR_NULL;
    if (g.workspace_bytes < pl.ws_bytes) return QGEMM_ERR_WORKSPACE;
    if (!aligned(g.workspace, 16)) return QGEMM_ERR_ALIGN;
  }
  const Extent out = extent3(g.out, num_tokens, g.out_token_stride, g.q_heads, g.out_head_stride, c->head_dim);
  const Extent others[] = {extent3(g.q, num_tokens, g.q_token_stride, g.q_heads, g.q_head_stride, c->head_dim),
                           cache_extent(c, c->k),
                           cache_extent(c, c->v),
                           extent(g.block_table, g.num_seqs * g.table_stride, 4),
                           extent(g.seq_lens, g.num_seqs, 4),
                           extent(q_start, g.num_seqs + 1, 4),
                           extent(pl.ws_bytes ? g.workspace : nullptr, (int64_t)pl.ws_bytes, 1)};
  for (const Extent& e : others)
    if (overlap(out, e)) return QGEMM_ERR_ALIAS;
  if (pl.ws_bytes)
    for (const Extent& e : others)
      if (&e != &others[6] && overlap(others[6], e)) return QGEMM_ERR_ALIAS;
  st = qg::check_current_device();
  if (st) return st;

  qg::AttnArgs a{};
  a.q = g.q;
  a.out = g.out;
  a.q_ts = g.q_token_stride;
  a.q_hs = g.q_head_stride;
  a.o_ts = g.out_token_stride;
  a.o_hs = g.out_head_stride;
  a.cache = cache_args(c, g.block_table, g.table_stride);
  a.lens = g.seq_lens;
  a.q_start = q_start;
  a.num_seqs = (int32_t)g.num_seqs;
  a.kv_heads = c->kv_heads;
  a.group = g.q_heads / c->kv_heads;
  a.head_dim = c->head_dim;
  a.num_tokens = (int32_t)num_tokens;
  a.max_q = (int32_t)max_q;
  a.max_len = (int32_t)g.max_len;
  a.window = (int32_t)mask.window;
  a.sinks = (int32_t)mask.sinks;
  a.row_tiles = pl.row_tiles;
  a.part_rows = pl.part_rows;
  a.splits = pl.splits;
  a.split_blocks = pl.split_blocks;
  a.inv_group = 1.0 / a.group;
  a.inv_kv_heads = 1.0 / a.kv_heads;
  a.inv_seqs = 1.0 / a.num_seqs;
  a.inv_heads = 1.0 / ((double)a.kv_heads * a.row_tiles);
  a.inv_tiles = 1.0 / (double)pl.tiles;
  a.scale_log2 = g.scale * c->k_scale * 1.44269504088896340736f;
  a.v_scale = c->v_scale;
  if (pl.ws_bytes) {
    char* ws = static_cast<char*>(g.workspace);
    a.counters = reinterpret_cast<uint32_t*>(ws);
    a.stats = reinterpret_cast<float*>(ws + pl.stats_offset);
    a.partial = reinterpret_cast<float*>(ws + pl.partial_offset);
  }
  const bool bf16 = g.act_dtype == QGEMM_DT_BF16, fp8 = c->dtype == QGEMM_DT_FP8;
  hipStream_t s = static_cast<hipStream_t>(g.stream);
  const hipError_t e = prefill ? qg::launch_attn_prefill(a, bf16, fp8, pl.tiles, s)
                               : qg::launch_attn_decode(a, bf16, fp8, pl.tiles, s);
  if (e != hipSuccess) return qg::fail_hip(e, "kernel launch");
  return QGEMM_OK;
}

int run_append(const qgemm_append_call& g) {
  const qgemm_kv_cache* c = g.cache;
  if (!c) return QGEMM_ERR_NULL;
  if (!valid_act(g.act_dtype) || (g.interleaved != 0 && g.interleaved != 1)) return QGEMM_ERR_RANGE;
  if (g.num_seqs < 0 || g.num_seqs > kMaxSeqs || g.num_tokens < 0 || g.num_tokens > kMaxTokens) return QGEMM_ERR_SHAPE;
  int st = check_cache(c, g.act_dtype);
  if (st) return st;
  st = check_heads(g.q_heads, c->kv_heads);
  if (st) return st;
  // 32-bit task numbers over the tokens' heads
  const int64_t heads = (int64_t)g.q_heads + 2 * c->kv_heads;
  if (g.num_tokens * heads >= (int64_t(1) << 31)) return QGEMM_ERR_SHAPE;
  if (g.rot_dim < 0 || g.rot_dim > c->head_dim || g.rot_dim % 16 != 0) return QGEMM_ERR_SHAPE;
  if (g.rope_rows < 0 || g.rope_rows > kMaxLen) return QGEMM_ERR_SHAPE;
  if (g.table_stride < 0 || g.table_stride > kMaxLen) return QGEMM_ERR_SHAPE;
  if ((g.q_norm || g.k_norm) && !(std::isfinite(g.eps) && g.eps >= 0.f)) return QGEMM_ERR_RANGE;
  if (g.num_tokens == 0) return QGEMM_OK;
  if (!g.q || !g.k || !g.v || !g.q_out || !g.positions || !g.block_table || (g.rot_dim > 0 && !g.rope))
    return QGEMM_ERR_NULL;
  for (const void* p : {g.q, g.k, g.v, g.q_norm, g.k_norm, (const void*)g.rope, (const void*)g.q_out})
    if (!aligned(p, 16)) return QGEMM_ERR_ALIGN;
  if (!aligned(g.positions, 4) || !aligned(g.token_seq, 4) || !aligned(g.block_table, 4)) return QGEMM_ERR_ALIGN;
  if (!valid_strides(g.num_tokens, g.q_token_stride, g.q_heads, g.q_head_stride, c->head_dim) ||
      !valid_strides(g.num_tokens, g.k_token_stride, c->kv_heads, g.k_head_stride, c->head_dim) ||
      !valid_strides(g.num_tokens, g.v_token_stride, c->kv_heads, g.v_head_stride, c->head_dim) ||
      !valid_out_strides(g.num_tokens, g.out_token_stride, g.q_heads, g.out_head_stride, c->head_dim))
    return QGEMM_ERR_ALIGN;
  const int64_t D = c->head_dim;
  const Extent eq = extent3(g.q, g.num_tokens, g.q_token_stride, g.q_heads, g.q_head_stride, D);
  const Extent out = extent3(g.q_out, g.num_tokens, g.out_token_stride, g.q_heads, g.out_head_stride, D);
  const Extent kc = cache_extent(c, c->k), vc = cache_extent(c, c->v);
  const Extent in[] = {extent3(g.k, g.num_tokens, g.k_token_stride, c->kv_heads, g.k_head_stride, D),
                       extent3(g.v, g.num_tokens, g.v_token_stride, c->kv_heads, g.v_head_stride, D),
                       extent(g.q_norm, D, 2),
                       extent(g.k_norm, D, 2),
                       extent(g.rope, g.rope_rows * g.rot_dim, 4),
                       extent(g.positions, g.num_tokens, 4),
                       extent(g.token_seq, g.num_tokens, 4),
                       extent(g.block_table, g.num_seqs * g.table_stride, 4)};
  const bool in_place =
      g.q_out == g.q && g.out_token_stride == g.q_token_stride && g.out_head_stride == g.q_head_stride;
  if (!in_place && overlap(out, eq)) return QGEMM_ERR_ALIAS;
  // the parts of one fused product interleave in memory: an in-place q_out may
  // span k and v without touching them, so only a separate q_out is checked
  for (const Extent& e : in)
    if ((!in_place && overlap(out, e)) || overlap(kc, e) || overlap(vc, e)) return QGEMM_ERR_ALIAS;
  if (overlap(kc, eq) || overlap(vc, eq) || overlap(kc, out) || overlap(vc, out)) return QGEMM_ERR_ALIAS;
  st = qg::check_current_device();
  if (st) return st;

  qg::AppendArgs a{};
  a.q = g.q;
  a.k = g.k;
  a.v = g.v;
  a.q_ts = g.q_token_stride;
  a.q_hs = g.q_head_stride;
  a.k_ts = g.k_token_stride;
  a.k_hs = g.k_head_stride;
  a.v_ts = g.v_token_stride;
  a.v_hs = g.v_head_stride;
  a.qo_ts = g.out_token_stride;
  a.qo_hs = g.out_head_stride;
  a.q_norm = g.q_norm;
  a.k_norm = g.k_norm;
  a.eps = g.eps;
  a.inv_dim = 1.0f / (float)c->head_dim;
  a.inv_heads = 1.0 / (double)heads;
  a.rope = g.rope;
  a.rope_rows = g.rope_rows;
  a.rot_dim = g.rot_dim;
  a.positions = g.positions;
  a.token_seq = g.token_seq;
  a.cache = cache_args(c, g.block_table, g.table_stride);
  a.num_seqs = (int32_t)g.num_seqs;
  a.num_tokens = (int32_t)g.num_tokens;
  a.q_heads = g.q_heads;
  a.kv_heads = c->kv_heads;
  a.head_dim = c->head_dim;
  a.q_out = g.q_out;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  const hipError_t e = qg::launch_append(a, g.act_dtype == QGEMM_DT_BF16, c->dtype == QGEMM_DT_FP8,
                                         g.interleaved != 0, static_cast<hipStream_t>(g.stream));
  if (e != hipSuccess) return qg::fail_hip(e, "kernel launch");
  return QGEMM_OK;
}

}  // namespace

extern "C" {

int qgemm_qk_rope_append_call(const qgemm_append_call* call) {
  return call ? run_append(*call) : QGEMM_ERR_NULL;
}

int qgemm_qk_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                         int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                         int64_t v_head_stride, const void* q_norm, const void* k_norm, float eps, const float* rope,
                         int64_t rope_rows, int32_t rot_dim, int32_t interleaved, const int32_t* positions,
                         const int32_t* token_seq, const int32_t* block_table, int64_t table_stride, int64_t num_seqs,
                         int64_t num_tokens, int32_t q_heads, int32_t act_dtype, const qgemm_kv_cache* cache,
                         void* q_out, int64_t qo_token_stride, int64_t qo_head_stride, void* stream) {
  qgemm_append_call g{};
  g.q = q;
  g.q_token_stride = q_token_stride;
  g.q_head_stride = q_head_stride;
  g.k = k;
  g.k_token_stride = k_token_stride;
  g.k_head_stride = k_head_stride;
  g.v = v;
  g.v_token_stride = v_token_stride;
  g.v_head_stride = v_head_stride;
  g.q_norm = q_norm;
  g.k_norm = k_norm;
  g.rope = rope;
  g.rope_rows = rope_rows;
  g.positions = positions;
  g.token_seq = token_seq;
  g.block_table = block_table;
  g.table_stride = table_stride;
  g.num_seqs = num_seqs;
  g.num_tokens = num_tokens;
  g.cache = cache;
  g.q_out = q_out;
  g.out_token_stride = qo_token_stride;
  g.out_head_stride = qo_head_stride;
  g.stream = stream;
  g.rot_dim = rot_dim;
  g.interleaved = interleaved;
  g.q_heads = q_heads;
  g.act_dtype = act_dtype;
  g.eps = eps;
  return run_append(g);
}

int qgemm_attn_decode_workspace_bytes(int64_t num_seqs, int64_t max_len, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim, int64_t window, int32_t sinks, size_t* bytes) {
  if (!bytes) return QGEMM_ERR_NULL;
  const int st = check_attn_shape(num_seqs, max_len, q_heads, kv_heads, head_dim, window, sinks);
  if (st) return st;
  const Mask mask = bounded_mask(max_len, window, sinks);
  *bytes = num_seqs == 0 ? 0 : decode_plan(num_seqs, max_len, q_heads, kv_heads, head_dim, mask).ws_bytes;
  return QGEMM_OK;
}

int qgemm_attn_decode_call(const qgemm_attn_call* call) {
  return call ? run_attn(*call, false) : QGEMM_ERR_NULL;
}

int qgemm_attn_decode(const void* q, int64_t q_token_stride, int64_t q_head_stride, const qgemm_kv_cache* cache,
                      const int32_t* block_table, int64_t table_stride, const int32_t* seq_lens, int64_t num_seqs,
                      int64_t max_len, int32_t q_heads, int32_t act_dtype, float scale, int64_t window, int32_t sinks,
                      void* out, int64_t out_token_stride, int64_t out_head_stride, void* workspace,
                      size_t workspace_bytes, void* stream) {
  qgemm_attn_call g{};
  g.q = q;
  g.q_token_stride = q_token_stride;
  g.q_head_stride = q_head_stride;
  g.cache = cache;
  g.block_table = block_table;
  g.table_stride = table_stride;
  g.seq_lens = seq_lens;
  g.num_seqs = num_seqs;
  g.max_len = max_len;
  g.window = window;
  g.out = out;
  g.out_token_stride = out_token_stride;
  g.out_head_stride = out_head_stride;
  g.workspace = workspace;
  g.workspace_bytes = workspace_bytes;
  g.stream = stream;
  g.q_heads = q_heads;
  g.act_dtype = act_dtype;
  g.sinks = sinks;
  g.scale = scale;
  return run_attn(g, false);
}

int qgemm_attn_prefill_workspace_bytes(int64_t num_seqs, int64_t max_q, int64_t max_len, int32_t q_heads,
                                       int32_t kv_heads, int32_t head_dim, int64_t window, int32_t sinks,
                                       size_t* bytes) {
  if (!bytes) return QGEMM_ERR_NULL;
  const int st = check_attn_shape(num_seqs, max_len, q_heads, kv_heads, head_dim, window, sinks);
  if (st) return st;
  if (max_q < 0 || max_q > kMaxTokens) return QGEMM_ERR_SHAPE;
  const Mask mask = bounded_mask(max_len, window, sinks);
  *bytes = num_seqs == 0 || max_q == 0
               ? 0
               : prefill_plan(num_seqs, max_q, max_len, q_heads, kv_heads, head_dim, mask).ws_bytes;
  return QGEMM_OK;
}

int qgemm_attn_prefill_call(const qgemm_attn_call* call) {
  return call ? run_attn(*call, true) : QGEMM_ERR_NULL;
}

int qgemm_attn_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride, const qgemm_kv_cache* cache,
                       const int32_t* block_table, int64_t table_stride, const int32_t* q_start,
                       const int32_t* seq_lens, int64_t num_seqs, int64_t num_tokens, int64_t max_q, int64_t max_len,
                       int32_t q_heads, int32_t act_dtype, float scale, int64_t window, int32_t sinks, void* out,
                       int64_t out_token_stride, int64_t out_head_stride, void* workspace, size_t workspace_bytes,
                       void* stream) {
  qgemm_attn_call g{};
  g.q = q;
  g.q_token_stride = q_token_stride;
  g.q_head_stride = q_head_stride;
  g.cache = cache;
  g.block_table = block_table;
  g.table_stride = table_stride;
  g.q_start = q_start;
  g.seq_lens = seq_lens;
  g.num_seqs = num_seqs;
  g.num_tokens = num_tokens;
  g.max_q = max_q;
  g.max_len = max_len;
  g.window = window;
  g.out = out;
  g.out_token_stride = out_token_stride;
  g.out_head_stride = out_head_stride;
  g.workspace = workspace;
  g.workspace_bytes = workspace_bytes;
  g.stream = stream;
  g.q_heads = q_heads;
  g.act_dtype = act_dtype;
  g.sinks = sinks;
  g.scale = scale;
  return run_attn(g, true);
}

int qgemm_attn_set_splits(int splits) {
  if (splits < 0 || splits > qg::kMaxAttnSplits) return QGEMM_ERR_RANGE;
  g_force_splits.store(splits);
  return QGEMM_OK;
}

}  // extern "C"
