// Launches of the many-token attention: the kernel of attn_prefill.h, and the join of a split length.
#include "attn_prefill.h"

namespace qg {
namespace {

// Joins the parts of the row tiles, in part order; a launch of its own, because the
// sums of 128 rows are more than the last workgroup of a tile can read at once. A
// thread takes four outputs of a row, `chunks` workgroups a tile.
template <class F>
__global__ void __launch_bounds__(256) attn_prefill_join(AttnArgs p, int chunks) {
  const int tile = (int)(blockIdx.x / (uint32_t)chunks);
  const RowTile rt = row_tile_of(p, tile);
  const int x = (blockIdx.x - tile * chunks) * 256 + threadIdx.x;
  const int quads = p.head_dim / 4;
  const int r = (int)((uint32_t)x / (uint32_t)quads), d = 4 * (x - r * quads);
  if (rt.parts == 1 || r >= rt.rows) return;
  constexpr int kBatch = 16;   // parts whose loads are in flight together
  float m = kNegInf, total = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < rt.parts; s0 += kBatch) {
    f32x4 y[kBatch];
    f32x2 ml[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t at = ((int64_t)tile * p.splits + min(s0 + u, rt.parts - 1)) * p.part_rows + r;
      y[u] = *reinterpret_cast<const f32x4*>(p.partial + at * p.head_dim + d);
      ml[u] = *reinterpret_cast<const f32x2*>(p.stats + 2 * at);
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) top = fmaxf(top, ml[u][0]);   // re-read last parts change nothing
    const float base = top == kNegInf ? 0.f : top;
    const float f0 = exp2_of(m - base);
    total *= f0;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= f0;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (s0 + u < rt.parts) {
        const float f = exp2_of(ml[u][0] - base);
        total += f * ml[u][1];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += f * y[u][i];
      }
    }
    m = top;
  }
  const int row = rt.row0 + r, qi = divide(row, p.inv_group);
  typename F::T* dst = static_cast<typename F::T*>(p.out) + (int64_t)(rt.q0 + qi) * p.o_ts +
                       (int64_t)(rt.kv_head * p.group + row - qi * p.group) * p.o_hs + d;
  *reinterpret_cast<u32x2*>(dst) = finish<F>(o, total, p.v_scale);
}

template <class F, class PF, bool FP8, int DP, int DU>
hipError_t launch_exact(const AttnArgs& a, int64_t tiles, hipStream_t s) {
  constexpr int lds = PrefillLds<DP>::kTotal;
  const hipError_t e = launch_in_runs(tiles * a.splits, [&](dim3 grid, uint32_t first) {
    AttnArgs r = a;
    r.first_block = first;
    if (DU == DP && a.head_dim == DP)
      hipLaunchKernelGGL((attn_prefill<F, PF, FP8, DP, DP, true>), grid, dim3(256), lds, s, r);
    else
      hipLaunchKernelGGL((attn_prefill<F, PF, FP8, DP, DU, false>), grid, dim3(256), lds, s, r);
  });
  if (e != hipSuccess || a.splits == 1) return e;
  // at most kMaxCounters tiles are split, in 32 chunks each: one launch
  static_assert(kMaxCounters * (kPrefillRows * kMaxHeadDim / 4 / 256) <= kMaxGrid, "the join's grid");
  const int chunks = (a.part_rows * (a.head_dim / 4) + 255) / 256;
  hipLaunchKernelGGL((attn_prefill_join<F>), dim3((unsigned)(tiles * chunks)), dim3(256), 0, s, a, chunks);
  return hipGetLastError();
}

// Heads of 65..96 and 129..192 values leave out a quarter of the products (4096 tokens,
// 32/8 heads, bf16: 96 values 138 -> 123 us, 80 133 -> 118, 192 321 -> 267).
template <class F, class PF, bool FP8>
hipError_t launch_dim(const AttnArgs& a, int64_t tiles, hipStream_t s) {
  if (a.head_dim <= 64) return launch_exact<F, PF, FP8, 64, 64>(a, tiles, s);
  if (a.head_dim <= 96) return launch_exact<F, PF, FP8, 128, 96>(a, tiles, s);
  if (a.head_dim <= 128) return launch_exact<F, PF, FP8, 128, 128>(a, tiles, s);
  if (a.head_dim <= 192) return launch_exact<F, PF, FP8, 256, 192>(a, tiles, s);
  return launch_exact<F, PF, FP8, 256, 256>(a, tiles, s);
}

}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s) {
  if (bf16) return fp8 ? launch_dim<BF16, F16, true>(a, tiles, s) : launch_dim<BF16, BF16, false>(a, tiles, s);
  return fp8 ? launch_dim<F16, F16, true>(a, tiles, s) : launch_dim<F16, F16, false>(a, tiles, s);
}

}  // namespace qg
