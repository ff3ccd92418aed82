// Host-side internals of the low-rank adapters: kernel arguments and launchers.
#pragma once

#include "qgemm.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qgemm_internal.h"

namespace qg {

constexpr int kLoraWaves = 4;         // waves of a workgroup
constexpr int kLoraRankTile = 16;     // ranks of one matrix product
constexpr int kLoraCols = 64;         // columns that a wave takes at a time
constexpr int kMaxLoraRank = 256;
constexpr int kMaxLoraAdapters = 4096;
constexpr int64_t kMaxLoraTokens = 65535;

// What the plan holds, in 32-bit words: a header (tokens, adapters, tiles of 16 rows, tiles of 64),
// the rows sorted by adapter (those without one last), and the tiles: runs of up to 16 and of up to
// 64 sorted rows of one adapter as (adapter or -1, first sorted row, rows, 0).
struct LoraPlanLayout {
  int64_t perm, tiles16, tiles64, words;   // offsets and size
  int64_t cap16, cap64;                    // most tiles
};
inline LoraPlanLayout lora_plan_layout(int64_t tokens, int64_t adapters) {
  LoraPlanLayout l;
  const int64_t runs = tokens < adapters + 1 ? tokens : adapters + 1;
  // a run of n rows takes at most n / 16 + 1 tiles, and no more than n
  l.cap16 = tokens < tokens / 16 + runs ? tokens : tokens / 16 + runs;
  l.cap64 = tokens < tokens / 64 + runs ? tokens : tokens / 64 + runs;
  l.perm = 16;
  l.tiles16 = (l.perm + tokens + 3) / 4 * 4;
  l.tiles64 = l.tiles16 + 4 * l.cap16;
  l.words = l.tiles64 + 4 * l.cap64;
  return l;
}

struct LoraPlanArgs {
  const int32_t* ids;
  int32_t* plan;
  int32_t tokens, adapters;
  int32_t tiles16, tiles64;   // offsets in words
};

struct LoraArgs {
  const void* x;
  const void* a;
  const void* b;
  const void* base;
  void* out;
  int64_t x_stride, base_stride, out_stride, a_stride, b_stride;
  const float* scales;
  const int32_t* ranks;
  const int32_t* plan;
  uint32_t* counters;     // one per tile and chunk, zero between calls
  float* partial;         // [tile][chunk][split], in fragment order
  float* y;               // [sorted row][slices][rank_tiles * 16]
  int32_t tokens, adapters, k, rank, slices;
  int32_t tiles16, tiles64;   // word offsets of the tiles in the plan
  int32_t cap16, cap64;       // most tiles
  int32_t tall_a, tall_b;     // tiles of 64 rows for the first, the second product (0: of 16)
  int32_t rank_tiles;     // of one slice
  int32_t splits, split_k;
  int32_t chunks;         // shrink: workgroups that share a tile's ranks
  int32_t group_cols;     // expand: 64-column tiles of a workgroup
  int32_t col_begin[QGEMM_LORA_MAX_SLICES + 1];   // first column of each slice
  int32_t group_begin[QGEMM_LORA_MAX_SLICES + 1]; // first workgroup of each slice
  int32_t in_place;       // rows without an adapter are left alone
};

struct LoraDecomposition {
  bool tall_a = false, tall_b = false;   // tiles of 64 rows (of 16) for the two products
  int rank_tiles = 1, chunk_tiles = 1, chunks = 1, splits = 1, split_k = 0;
  size_t y_offset = 0, partial_offset = 0, ws_bytes = 0;
};

hipError_t launch_lora_plan(const LoraPlanArgs& a, hipStream_t s);
hipError_t launch_lora_shrink(const LoraArgs& a, bool bf16, int chunk_tiles, hipStream_t s);
hipError_t launch_lora_expand(const LoraArgs& a, bool bf16, hipStream_t s);

}  // namespace qg
