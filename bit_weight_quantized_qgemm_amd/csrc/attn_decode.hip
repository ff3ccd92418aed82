// Launches of the one-token attention (attn_decode.h).
#include "attn_decode.h"

namespace qg {
namespace {

template <class F, class PF, bool FP8, int DP>
hipError_t launch_exact(const AttnArgs& a, int64_t tiles, hipStream_t s) {
  return launch_in_runs(tiles * a.splits, [&](dim3 grid, uint32_t first) {
    AttnArgs r = a;
    r.first_block = first;
    if (a.head_dim == DP) hipLaunchKernelGGL((attn_decode<F, PF, FP8, DP, true>), grid, dim3(256), 0, s, r);
    else hipLaunchKernelGGL((attn_decode<F, PF, FP8, DP, false>), grid, dim3(256), 0, s, r);
  });
}

template <class F, class PF, bool FP8>
hipError_t launch_dim(const AttnArgs& a, int64_t tiles, hipStream_t s) {
  if (a.head_dim <= 64) return launch_exact<F, PF, FP8, 64>(a, tiles, s);
  if (a.head_dim <= 128) return launch_exact<F, PF, FP8, 128>(a, tiles, s);
  return launch_exact<F, PF, FP8, 256>(a, tiles, s);
}

}  // namespace

// Against an e4m3 cache the weights and values meet in fp16 for both activation
// types: every e4m3 code is exact there, and the weights (at most 2^8) keep 11
// bits instead of 8.
hipError_t launch_attn_decode(const AttnArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s) {
  if (bf16) return fp8 ? launch_dim<BF16, F16, true>(a, tiles, s) : launch_dim<BF16, BF16, false>(a, tiles, s);
  return fp8 ? launch_dim<F16, F16, true>(a, tiles, s) : launch_dim<F16, F16, false>(a, tiles, s);
}

}  // namespace qg
