// Host-side internals of the attention operators: kernel arguments and launchers.
#pragma once

#include "qgemm.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qgemm_internal.h"

namespace qg {

// Tokens are handled in blocks of 16 (a page holds whole blocks, so a block has
// one page).
constexpr int kTokBlock = 16;
// A decode workgroup's waves take pairs of token blocks in turn.
constexpr int kDecodeWaves = 4;
constexpr int kDecodeRows = 16;       // query heads of one workgroup (MFMA columns)
constexpr int kPrefillRows = 128;     // rows (heads of tokens) of one workgroup
constexpr int kMaxHeadDim = 256;
constexpr int kMaxAttnSplits = 1024;
// A launch has fewer than 2^32 threads: grids of 256-thread workgroups above this many
// go out as several launches, each telling its first workgroup's number.
constexpr int64_t kMaxGrid = int64_t(1) << 23;
template <class Launch>
hipError_t launch_in_runs(int64_t workgroups, const Launch& launch) {
  for (int64_t first = 0; first < workgroups; first += kMaxGrid) {
    launch(dim3((unsigned)(workgroups - first < kMaxGrid ? workgroups - first : kMaxGrid)), (uint32_t)first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The cache as the kernels see it. `magic` divides a block number (below 2^20)
// by page_blocks (at most 2^12): n / d = (n * magic) >> 32 with
// magic = ceil(2^32 / d), exact because n * (magic * d - 2^32) < 2^32; 0 stands
// for d = 1.
struct CacheArgs {
  const void* k;
  const void* v;
  int64_t page_stride, token_stride, head_stride;   // elements
  const int32_t* table;
  int64_t table_stride;
  int32_t num_pages;
  int32_t page_blocks;
  uint32_t magic;
};

struct AttnArgs {
  const void* q;
  void* out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  CacheArgs cache;
  const int32_t* lens;
  const int32_t* q_start;   // prefill
  float* partial;           // [tile][split][part_rows][head_dim], sums before the division
                            // (own tokens beside shared ones, many-token calls: as shared_partial)
  float* stats;             // [tile][split][part_rows] (maximum in log2 units, sum of weights)
  uint32_t* counters;       // decode: one per tile, zero between calls
  int32_t num_seqs, kv_heads, group, head_dim;
  int32_t num_tokens, max_q, max_len;   // prefill; prefill; both
  int32_t window, sinks;
  int32_t row_tiles;        // row tiles per (sequence, key-value head)
  int32_t part_rows;        // rows of a tile that the partial sums hold
  int32_t splits;           // most parts of a row tile
  int32_t split_blocks;     // token blocks of a part
  double inv_group, inv_kv_heads, inv_seqs, inv_heads, inv_tiles;   // 1 / group, ... (heads: row tiles of a sequence)
  float scale_log2;         // scale * k_scale * log2(e)
  float v_scale;
  uint32_t first_block;     // number of the launch's first workgroup
};

// The same for a batch whose sequences share their first tokens group by group:
// sequences group_start[g]..group_start[g+1]-1 the first shared_lens[g] ones.
struct SharedArgs : AttnArgs {
  const int32_t* group_start;
  const int32_t* shared_lens;
  float* shared_partial;    // [shared split][kv head][token][head of it][head_dim]
  float* shared_stats;      // [shared split][kv head][token][head of it] (maximum, sum)
  int32_t num_groups, max_shared;
  int32_t shared_splits;
  int32_t shared_split_blocks;   // token blocks of a part
  int32_t shared_blocks;    // workgroups of the shared tokens: the first ones of the launch
  int32_t split_step;       // token blocks of an own part: a multiple of this
  int32_t own_parts, own_part_blocks;   // of a sequence with the own tokens that the plan counts on
  double inv_shared_splits;
};

struct AttnPlan {
  int64_t tiles = 0;        // row tiles of the launch
  int row_tiles = 1;        // per (sequence, key-value head)
  int part_rows = 0;
  int splits = 1;
  int split_blocks = 0;
  size_t stats_offset = 0, partial_offset = 0, ws_bytes = 0;   // 0 bytes when unsplit
};

struct AppendArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs;
  const void* q_norm;
  const void* k_norm;
  float eps, inv_dim;
  double inv_heads;   // 1 / (q_heads + 2 kv_heads)
  const float* rope;
  int64_t rope_rows;
  int32_t rot_dim;
  const int32_t* positions;
  const int32_t* token_seq;
  CacheArgs cache;
  int32_t num_seqs, num_tokens, q_heads, kv_heads, head_dim;
  void* q_out;
  float k_scale, v_scale;
  uint32_t first_block;   // number of the launch's first workgroup
};

// Workspace of a batch with shared tokens: the own parts', then the shared ones'.
struct SharedPlan {
  AttnPlan own;
  bool share = false;       // false: computed as if nothing were shared
  int own_parts = 1, own_part_blocks = 0;
  int64_t tiles = 0;        // of shared rows
  int splits = 1;
  int split_blocks = 1;
  size_t stats_offset = 0, partial_offset = 0, ws_bytes = 0;
};

hipError_t launch_append(const AppendArgs& a, bool bf16, bool fp8, bool interleaved, hipStream_t s);
hipError_t launch_attn_decode(const AttnArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s);
hipError_t launch_attn_prefill(const AttnArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s);
// The same for a batch with shared tokens (tiles: of the own ones).
hipError_t launch_attn_decode_shared(const SharedArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s);
hipError_t launch_attn_prefill_shared(const SharedArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s);

}  // namespace qg
