// Attention of one new token per sequence on the tokens that it shares with no other, joined
// with what attn_shared.hip left of the shared ones.
#include "attn_decode.h"

namespace qg {
namespace {

template <class F, class PF, bool FP8, int DP>
hipError_t launch_exact(const SharedArgs& a, int64_t tiles, hipStream_t s) {
  return launch_in_runs(tiles * a.splits, [&](dim3 grid, uint32_t first) {
    SharedArgs r = a;
    r.first_block = first;
    if (a.head_dim == DP) hipLaunchKernelGGL((attn_decode_own<F, PF, FP8, DP, true>), grid, dim3(256), 0, s, r);
    else hipLaunchKernelGGL((attn_decode_own<F, PF, FP8, DP, false>), grid, dim3(256), 0, s, r);
  });
}

template <class F, class PF, bool FP8>
hipError_t launch_dim(const SharedArgs& a, int64_t tiles, hipStream_t s) {
  if (a.head_dim <= 64) return launch_exact<F, PF, FP8, 64>(a, tiles, s);
  if (a.head_dim <= 128) return launch_exact<F, PF, FP8, 128>(a, tiles, s);
  return launch_exact<F, PF, FP8, 256>(a, tiles, s);
}

}  // namespace

hipError_t launch_attn_decode_own(const SharedArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s) {
  if (bf16) return fp8 ? launch_dim<BF16, F16, true>(a, tiles, s) : launch_dim<BF16, BF16, false>(a, tiles, s);
  return fp8 ? launch_dim<F16, F16, true>(a, tiles, s) : launch_dim<F16, F16, false>(a, tiles, s);
}

}  // namespace qg
