// Several new tokens per sequence over shared and own tokens, and the join of both.
#include "attn_shared_parts.h"

namespace qg {
namespace {

// A thread takes four outputs of a row at a time, `chunks` workgroups a tile of rows: its own
// parts in order, then the shared ones. 16 x 5 rows of 64 heads on 6000 shared tokens in 6
// parts: 7 us.
template <class F>
__global__ void __launch_bounds__(256) attn_join_many(SharedArgs p, int chunks) {
  const uint32_t block = blockIdx.x + p.first_block;
  const int tile = (int)(block / (uint32_t)chunks), chunk = (int)(block - (uint32_t)tile * (uint32_t)chunks);
  const RowTile rt = own_tile_of(p, tile);
  if (rt.rows <= 0) return;
  const int shared = shared_tokens(p, rt.seq);
  const int quads = p.head_dim / 4;
  for (int x = chunk * 256 + threadIdx.x; x < rt.rows * quads; x += chunks * 256) {
    const int r = x / quads, d = 4 * (x - r * quads);
    RowSums sums;
    const int row = rt.row0 + r, qi = divide(row, p.inv_group), token = rt.q0 + qi;
    const int head = rt.kv_head * p.group + row - qi * p.group;
    add_parts(sums, rt.parts, [&](int s, f32x4& y, float& m, float& l) {
      const int64_t at = part_place(p, s, rt.kv_head, rt.q0 * p.group + row);
      y = *reinterpret_cast<const f32x4*>(p.partial + at * p.head_dim + d);
      const f32x2 ml = *reinterpret_cast<const f32x2*>(p.stats + 2 * at);
      m = ml[0];
      l = ml[1];
    });
    add_shared_parts(sums, p, shared, rt.kv_head, rt.q0 * p.group + row, d);
    typename F::T* dst = static_cast<typename F::T*>(p.out) + (int64_t)token * p.o_ts + (int64_t)head * p.o_hs + d;
    *reinterpret_cast<u32x2*>(dst) = finish<F>(sums.o, sums.total, p.v_scale);
  }
}

}  // namespace

hipError_t launch_attn_prefill_shared(const SharedArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s) {
  const hipError_t e = launch_parts<false>(a, bf16, fp8, tiles, s);
  if (e != hipSuccess) return e;
  // four turns of a workgroup where the tiles alone fill the device
  const int all = (a.part_rows * (a.head_dim / 4) + 255) / 256, chunks = tiles >= 1024 ? (all + 3) / 4 : all;
  return launch_in_runs(tiles * chunks, [&](dim3 grid, uint32_t first) {
    SharedArgs r = a;
    r.first_block = first;
    if (bf16) hipLaunchKernelGGL((attn_join_many<BF16>), grid, dim3(256), 0, s, r, chunks);
    else hipLaunchKernelGGL((attn_join_many<F16>), grid, dim3(256), 0, s, r, chunks);
  });
}

}  // namespace qg
