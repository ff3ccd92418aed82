// Attention of a group's rows on the tokens that its sequences share: the kernel of
// attn_prefill.h with the rows of all sequences of a group as one tile after the other.
#include "attn_prefill.h"

namespace qg {
namespace {

template <class F, class PF, bool FP8, int DP, int DU>
hipError_t launch_exact(const SharedArgs& a, hipStream_t s) {
  constexpr int lds = PrefillLds<DP>::kTotal;
  return launch_in_runs((int64_t)a.shared_tiles * a.shared_splits, [&](dim3 grid, uint32_t first) {
    SharedArgs r = a;
    r.first_block = first;
    if (DU == DP && a.head_dim == DP)
      hipLaunchKernelGGL((attn_prefill_part<F, PF, FP8, DP, DP, true, kShared>), grid, dim3(256), lds, s, r);
    else
      hipLaunchKernelGGL((attn_prefill_part<F, PF, FP8, DP, DU, false, kShared>), grid, dim3(256), lds, s, r);
  });
}

template <class F, class PF, bool FP8>
hipError_t launch_dim(const SharedArgs& a, hipStream_t s) {
  if (a.head_dim <= 64) return launch_exact<F, PF, FP8, 64, 64>(a, s);
  if (a.head_dim <= 96) return launch_exact<F, PF, FP8, 128, 96>(a, s);
  if (a.head_dim <= 128) return launch_exact<F, PF, FP8, 128, 128>(a, s);
  if (a.head_dim <= 192) return launch_exact<F, PF, FP8, 256, 192>(a, s);
  return launch_exact<F, PF, FP8, 256, 256>(a, s);
}

}  // namespace

hipError_t launch_attn_shared(const SharedArgs& a, bool bf16, bool fp8, hipStream_t s) {
  if (bf16) return fp8 ? launch_dim<BF16, F16, true>(a, s) : launch_dim<BF16, BF16, false>(a, s);
  return fp8 ? launch_dim<F16, F16, true>(a, s) : launch_dim<F16, F16, false>(a, s);
}

}  // namespace qg
