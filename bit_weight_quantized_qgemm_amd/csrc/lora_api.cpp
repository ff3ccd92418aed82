// C-ABI front end of the low-rank adapters: argument validation (before any HIP
// call), the work decomposition and kernel dispatch. See include/qgemm.h for the
// contract.
#include "qgemm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora_internal.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 32;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A tensor's bytes in memory: [first, last).
struct Extent {
  uintptr_t first = 0, last = 0;
};
bool overlap(const Extent& a, const Extent& b) { return a.first < b.last && b.first < a.last; }
Extent extent(const void* p, int64_t elems, int64_t elt) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return p && elems > 0 ? Extent{a, a + (uintptr_t)(elems * elt)} : Extent{};
}
Extent extent2(const void* p, int64_t rows, int64_t stride, int64_t cols) {
  return extent(p, (rows - 1) * stride + cols, 2);
}

int check_counts(int64_t num_tokens, int64_t num_adapters) {
  if (num_tokens < 0 || num_tokens > qg::kMaxLoraTokens) return QGEMM_ERR_SHAPE;
  if (num_adapters < 1 || num_adapters > qg::kMaxLoraAdapters) return QGEMM_ERR_SHAPE;
  return QGEMM_OK;
}

int check_shape(int64_t K, int64_t N, int32_t rank, int32_t slices) {
  if (K < 8 || K > kMaxDim || K % 8 != 0 || N < 8 || N > kMaxDim || N % 8 != 0) return QGEMM_ERR_SHAPE;
  if (rank < 8 || rank > qg::kMaxLoraRank || rank % 8 != 0) return QGEMM_ERR_SHAPE;
  if (slices < 1 || slices > QGEMM_LORA_MAX_SLICES) return QGEMM_ERR_SHAPE;
  return QGEMM_OK;
}

// A stride of rows of `cols` elements; not used where there is one row.
bool valid_stride(int64_t rows, int64_t stride, int64_t cols) {
  return rows == 1 || (stride >= cols && stride <= kMaxStride && stride % 8 == 0);
}

qg::LoraDecomposition decompose(int64_t tokens, int64_t adapters, int64_t K, int32_t rank, int32_t slices) {
  qg::LoraDecomposition d;
  const qg::LoraPlanLayout l = qg::lora_plan_layout(tokens, adapters);
  // Tiles of 64 rows read the adapter's matrices once for four times the rows, tiles of 16
  // leave more workgroups and fewer empty rows. Measured, us (16 / 64 rows; 4096 to 11008,
  // five adapters unless stated):
  //  - A x: 1003 rows, rank 64 10.3 / 15.6; 1500 of 8192 values, rank 32 15.4 / 13.8; 2048,
  //    rank 64 18.6 / 16.0, rank 16 9.9 / 9.3; 4096, rank 128 55.5 / 31.4.
  //  - its product with B, ranks above 32: 512 rows of 40 adapters 18.1 / 21.5, 1003 rows
  //    23.3 / 21.7, 2048 40.1 / 36.9, 4096, rank 128 127 / 76; ranks to 32, whose B is
  //    little: 1500 rows 19.3 / 21.4, 2048 20.8 / 25.6, 8192 to 8192 columns 61 / 55.
  d.tall_a = tokens > 1024;
  d.tall_b = tokens > (rank > 32 ? 768 : 2560);
  const int64_t cap = d.tall_a ? l.cap64 : l.cap16;
  d.rank_tiles = (rank + qg::kLoraRankTile - 1) / qg::kLoraRankTile;
  const int64_t tiles = (int64_t)slices * d.rank_tiles;
  d.chunks = (int)((tiles + 3) / 4);   // of up to four tiles, whose sums stay in registers
  d.chunk_tiles = (int)((tiles + d.chunks - 1) / d.chunks);
  // Parts of K, in whole units (a run of steps for each of a workgroup's four waves).
  //  - Tiles of 16 rows: up to two workgroups per compute unit, of equal length (48 ranks on
  //    8192, us: 64 rows of 64 adapters in 4 parts 12.9, 6 14.7, 8 12.2, 16 16.7; 256 rows of 60
  //    in 4, 6, 8 12.9, 15.4, 12.6; 128 rows of 24 at rank 64 in 4 13.9, 8 9.6, 16 10.8).
  //  - Tiles of 64 rows: the fewest turns of the units, a turn counting its length and one
  //    more (8192 rows of 8192, rank 16: 134 tiles in 1, 2, 3, 4, 5 parts 47, 57, 41, 49, 43;
  //    of 4096 at 96 ranks, 266 in 1, 2, 4, 6: 55, 47, 45, 50; 2048 of 8192 at rank 32, 38 in
  //    1, 4, 6, 8: 46, 17.5, 15.3, 17.9).
  // More tiles than the workspace has counters fill the device without parts.
  const int64_t unit = d.tall_a ? 256 : 512, units = (K + unit - 1) / unit, cus = qg::device_cu_count();
  int64_t per = units;   // units of a part
  if (cap * d.chunks > qg::kMaxCounters) {
  } else if (d.tall_a) {
    int64_t least = INT64_MAX;
    for (int64_t s = 1; s <= std::min<int64_t>(units, 8); ++s) {
      const int64_t each = (units + s - 1) / s, cost = (cap * d.chunks * s + cus - 1) / cus * (each + 1);
      if (cost < least) least = cost, per = each;
    }
  } else {
    const int64_t want = std::max<int64_t>(1, 2 * cus / std::max<int64_t>(1, cap * d.chunks));
    const int64_t fewest = (units + want - 1) / want;
    per = fewest;
    while (units % per != 0 && per < 2 * fewest) ++per;
  }
  d.split_k = (int)(per * unit);
  d.splits = (int)((K + d.split_k - 1) / d.split_k);
  d.y_offset = qg::kCounterBytes;
  d.partial_offset = d.y_offset + qg::align256((size_t)tokens * tiles * 16 * 4);
  const size_t part = (size_t)(d.tall_a ? 4 : 1) * d.chunk_tiles * 1024;
  d.ws_bytes = d.partial_offset + (d.splits > 1 ? (size_t)(cap * d.chunks * d.splits) * part : 0);
  return d;
}

int run_lora(const qgemm_lora_call& g) {
  const qgemm_lora_adapters* w = g.adapters;
  if (!w) return QGEMM_ERR_NULL;
  if (w->dtype != QGEMM_DT_F16 && w->dtype != QGEMM_DT_BF16) return QGEMM_ERR_RANGE;
  int st = check_counts(g.num_tokens, w->num_adapters);
  if (st) return st;
  st = check_shape(w->K, w->N, w->rank, w->slices);
  if (st) return st;
  int64_t columns = 0;
  for (int i = 0; i < w->slices; ++i) {
    if (w->widths[i] < 8 || w->widths[i] > w->N || w->widths[i] % 8 != 0) return QGEMM_ERR_SHAPE;
    columns += w->widths[i];
  }
  if (columns != w->N) return QGEMM_ERR_SHAPE;
  if (!w->a || !w->b) return QGEMM_ERR_NULL;
  if (!aligned(w->a, 16) || !aligned(w->b, 16) || !aligned(w->scales, 4) || !aligned(w->ranks, 4)) return QGEMM_ERR_ALIGN;
  const int64_t a_elems = (int64_t)w->slices * w->rank * w->K, b_elems = w->N * w->rank;
  if (!valid_stride(w->num_adapters, w->a_stride, a_elems) || !valid_stride(w->num_adapters, w->b_stride, b_elems))
    return QGEMM_ERR_ALIGN;
  if (g.num_tokens == 0) return QGEMM_OK;
  if (!g.x || !g.out || !g.plan) return QGEMM_ERR_NULL;
  if (!aligned(g.x, 16) || !aligned(g.out, 16) || !aligned(g.base, 16) || !aligned(g.plan, 16)) return QGEMM_ERR_ALIGN;
  if (!valid_stride(g.num_tokens, g.x_stride, w->K) || !valid_stride(g.num_tokens, g.out_stride, w->N) ||
      (g.base && !valid_stride(g.num_tokens, g.base_stride, w->N)))
    return QGEMM_ERR_ALIGN;
  const qg::LoraPlanLayout l = qg::lora_plan_layout(g.num_tokens, w->num_adapters);
  if (g.plan_bytes != (size_t)l.words * 4) return QGEMM_ERR_SIZE;
  const qg::LoraDecomposition d = decompose(g.num_tokens, w->num_adapters, w->K, w->rank, w->slices);
  if (!g.workspace) return QGEMM_ERR_NULL;
  if (g.workspace_bytes < d.ws_bytes) return QGEMM_ERR_WORKSPACE;
  if (!aligned(g.workspace, 16)) return QGEMM_ERR_ALIGN;
  const Extent out = extent2(g.out, g.num_tokens, g.out_stride, w->N);
  const Extent base = extent2(g.base, g.num_tokens, g.base_stride, w->N);
  const Extent ws = extent(g.workspace, (int64_t)d.ws_bytes, 1);
  const bool in_place = g.base == g.out && (g.num_tokens == 1 || g.base_stride == g.out_stride);
  if (g.base && !in_place && overlap(out, base)) return QGEMM_ERR_ALIAS;
  const Extent others[] = {extent2(g.x, g.num_tokens, g.x_stride, w->K),
                           extent2(w->a, w->num_adapters, w->a_stride, a_elems),
                           extent2(w->b, w->num_adapters, w->b_stride, b_elems),
                           extent(w->scales, w->num_adapters, 4),
                           extent(w->ranks, w->num_adapters, 4),
                           extent(g.plan, (int64_t)g.plan_bytes, 1)};
  for (const Extent& e : others)
    if (overlap(out, e) || overlap(ws, e)) return QGEMM_ERR_ALIAS;
  if (overlap(ws, out) || overlap(ws, base)) return QGEMM_ERR_ALIAS;
  st = qg::check_current_device();
  if (st) return st;

  qg::LoraArgs a{};
  a.x = g.x;
  a.a = w->a;
  a.b = w->b;
  a.base = g.base;
  a.out = g.out;
  a.x_stride = g.x_stride;
  a.base_stride = g.base_stride;
  a.out_stride = g.out_stride;
  a.a_stride = w->a_stride;
  a.b_stride = w->b_stride;
  a.scales = w->scales;
  a.ranks = w->ranks;
  a.plan = static_cast<const int32_t*>(g.plan);
  char* ws_base = static_cast<char*>(g.workspace);
  a.counters = reinterpret_cast<uint32_t*>(ws_base);
  a.y = reinterpret_cast<float*>(ws_base + d.y_offset);
  a.partial = reinterpret_cast<float*>(ws_base + d.partial_offset);
  a.tokens = (int32_t)g.num_tokens;
  a.adapters = w->num_adapters;
  a.k = (int32_t)w->K;
  a.rank = w->rank;
  a.slices = w->slices;
  a.tiles16 = (int32_t)l.tiles16;
  a.tiles64 = (int32_t)l.tiles64;
  a.cap16 = (int32_t)l.cap16;
  a.cap64 = (int32_t)l.cap64;
  a.tall_a = d.tall_a;
  a.tall_b = d.tall_b;
  a.rank_tiles = d.rank_tiles;
  a.splits = d.splits;
  a.split_k = d.split_k;
  a.chunks = d.chunks;
  a.in_place = g.base && in_place;
  // Columns: a wave takes one tile of 64, two where that leaves 16 waves per compute unit
  // (8192 rows, 8192 to 8192, rank 16: one 58 us, two 55, four 60; 64 rows of 64 adapters
  // 9.4, 7.7, 8.6); more where the grid would pass 2^20 workgroups.
  const int64_t col_tiles = (w->N + qg::kLoraCols - 1) / qg::kLoraCols;
  int64_t each = std::max<int64_t>(1, std::min<int64_t>((d.tall_b ? l.cap64 : l.cap16) * col_tiles / (16 * qg::device_cu_count()), 2));
  while (l.cap16 * (col_tiles / (qg::kLoraWaves * each) + w->slices) > (int64_t(1) << 20)) each *= 2;
  a.group_cols = (int32_t)(qg::kLoraWaves * each);
  for (int i = 0; i < w->slices; ++i) {
    const int64_t tiles = (w->widths[i] + qg::kLoraCols - 1) / qg::kLoraCols;
    a.col_begin[i + 1] = a.col_begin[i] + (int32_t)w->widths[i];
    a.group_begin[i + 1] = a.group_begin[i] + (int32_t)((tiles + a.group_cols - 1) / a.group_cols);
  }
  const bool bf16 = w->dtype == QGEMM_DT_BF16;
  hipStream_t s = static_cast<hipStream_t>(g.stream);
  hipError_t e = qg::launch_lora_shrink(a, bf16, d.chunk_tiles, s);
  if (e == hipSuccess) e = qg::launch_lora_expand(a, bf16, s);
  if (e != hipSuccess) return qg::fail_hip(e, "kernel launch");
  return QGEMM_OK;
}

}  // namespace

extern "C" {

int qgemm_lora_plan_bytes(int64_t num_tokens, int64_t num_adapters, size_t* bytes) {
  if (!bytes) return QGEMM_ERR_NULL;
  const int st = check_counts(num_tokens, num_adapters);
  if (st) return st;
  *bytes = (size_t)qg::lora_plan_layout(num_tokens, num_adapters).words * 4;
  return QGEMM_OK;
}

int qgemm_lora_plan(const int32_t* ids, int64_t num_tokens, int64_t num_adapters, void* plan, size_t plan_bytes,
                    void* stream) {
  int st = check_counts(num_tokens, num_adapters);
  if (st) return st;
  if (num_tokens == 0) return QGEMM_OK;
  if (!ids || !plan) return QGEMM_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(plan, 16)) return QGEMM_ERR_ALIGN;
  const qg::LoraPlanLayout l = qg::lora_plan_layout(num_tokens, num_adapters);
  if (plan_bytes != (size_t)l.words * 4) return QGEMM_ERR_SIZE;
  if (overlap(extent(ids, num_tokens, 4), extent(plan, (int64_t)plan_bytes, 1))) return QGEMM_ERR_ALIAS;
  st = qg::check_current_device();
  if (st) return st;
  qg::LoraPlanArgs a{};
  a.ids = ids;
  a.plan = static_cast<int32_t*>(plan);
  a.tokens = (int32_t)num_tokens;
  a.adapters = (int32_t)num_adapters;
  a.tiles16 = (int32_t)l.tiles16;
  a.tiles64 = (int32_t)l.tiles64;
  const hipError_t e = qg::launch_lora_plan(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return qg::fail_hip(e, "kernel launch");
  return QGEMM_OK;
}

int qgemm_lora_workspace_bytes(int64_t num_tokens, int64_t num_adapters, int64_t K, int64_t N, int32_t rank,
                               int32_t slices, size_t* bytes) {
  if (!bytes) return QGEMM_ERR_NULL;
  int st = check_counts(num_tokens, num_adapters);
  if (st) return st;
  st = check_shape(K, N, rank, slices);
  if (st) return st;
  *bytes = num_tokens == 0 ? 0 : decompose(num_tokens, num_adapters, K, rank, slices).ws_bytes;
  return QGEMM_OK;
}

int qgemm_lora(const qgemm_lora_call* call) { return call ? run_lora(*call) : QGEMM_ERR_NULL; }

}  // extern "C"
