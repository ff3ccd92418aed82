// Attention of several new tokens per sequence on the tokens that it shares with no other, and
// its join with what attn_shared.hip left of the shared ones.
#include "attn_prefill.h"

namespace qg {
namespace {

// A thread takes four outputs of a row, `chunks` workgroups a tile: the own parts in order, then
// the shared ones.
template <class F>
__global__ void __launch_bounds__(256) attn_join_shared(SharedArgs p, int chunks) {
  const uint32_t block = blockIdx.x + p.first_block;
  const int tile = (int)(block / (uint32_t)chunks);
  const RowTile rt = own_tile_of(p, tile);
  const int x = (int)(block - (uint32_t)(tile * chunks)) * 256 + threadIdx.x;
  const int quads = p.head_dim / 4;
  const int r = (int)((uint32_t)x / (uint32_t)quads), d = 4 * (x - r * quads);
  if (rt.rows <= 0) return;
  const SharedGroup g = group_of(p, rt.seq);
  if (r >= rt.rows) return;
  RowSums sums;
  const int64_t first = (int64_t)tile * p.splits * p.part_rows + r;
  add_parts(sums, rt.parts, [&](int s, f32x4& y, float& m, float& l) {
    const int64_t at = first + (int64_t)s * p.part_rows;
    y = *reinterpret_cast<const f32x4*>(p.partial + at * p.head_dim + d);
    const f32x2 ml = *reinterpret_cast<const f32x2*>(p.stats + 2 * at);
    m = ml[0];
    l = ml[1];
  });
  const int row = rt.row0 + r, qi = divide(row, p.inv_group), head = row - qi * p.group;
  add_shared_parts(sums, p, g, rt.kv_head, rt.q0 + qi - token_of(p, g.seq), head, d);
  typename F::T* dst = static_cast<typename F::T*>(p.out) + (int64_t)(rt.q0 + qi) * p.o_ts +
                       (int64_t)(rt.kv_head * p.group + head) * p.o_hs + d;
  *reinterpret_cast<u32x2*>(dst) = finish<F>(sums.o, sums.total, p.v_scale);
}

template <class F, class PF, bool FP8, int DP, int DU>
hipError_t launch_exact(const SharedArgs& a, int64_t tiles, hipStream_t s) {
  constexpr int lds = PrefillLds<DP>::kTotal;
  hipError_t e = launch_in_runs(tiles * a.splits, [&](dim3 grid, uint32_t first) {
    SharedArgs r = a;
    r.first_block = first;
    if (DU == DP && a.head_dim == DP)
      hipLaunchKernelGGL((attn_prefill_part<F, PF, FP8, DP, DP, true, kOwn>), grid, dim3(256), lds, s, r);
    else
      hipLaunchKernelGGL((attn_prefill_part<F, PF, FP8, DP, DU, false, kOwn>), grid, dim3(256), lds, s, r);
  });
  if (e != hipSuccess) return e;
  const int chunks = (a.part_rows * (a.head_dim / 4) + 255) / 256;
  return launch_in_runs(tiles * chunks, [&](dim3 grid, uint32_t first) {
    SharedArgs r = a;
    r.first_block = first;
    hipLaunchKernelGGL((attn_join_shared<F>), grid, dim3(256), 0, s, r, chunks);
  });
}

template <class F, class PF, bool FP8>
hipError_t launch_dim(const SharedArgs& a, int64_t tiles, hipStream_t s) {
  if (a.head_dim <= 64) return launch_exact<F, PF, FP8, 64, 64>(a, tiles, s);
  if (a.head_dim <= 96) return launch_exact<F, PF, FP8, 128, 96>(a, tiles, s);
  if (a.head_dim <= 128) return launch_exact<F, PF, FP8, 128, 128>(a, tiles, s);
  if (a.head_dim <= 192) return launch_exact<F, PF, FP8, 256, 192>(a, tiles, s);
  return launch_exact<F, PF, FP8, 256, 256>(a, tiles, s);
}

}  // namespace

hipError_t launch_attn_prefill_own(const SharedArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s) {
  if (bf16) return fp8 ? launch_dim<BF16, F16, true>(a, tiles, s) : launch_dim<BF16, BF16, false>(a, tiles, s);
  return fp8 ? launch_dim<F16, F16, true>(a, tiles, s) : launch_dim<F16, F16, false>(a, tiles, s);
}

}  // namespace qg
