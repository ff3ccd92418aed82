// Attention for a batch whose sequences share their first tokens, group by group: one launch
// computes the shared tokens for all rows of a group (the many-token kernel of
// attn_prefill.h) and each sequence's own tokens (that kernel, or the one-token kernel of
// attn_decode.h), a second joins both.
//
// The two kinds of workgroups run side by side because they are bound by different things:
// the shared tokens' by the matrix units, with as many rows as the group has, the own tokens'
// by the stream of the cache. The shared ones come first and are cut into about one
// workgroup per compute unit, which leaves room for one of the others beside it.
//
// Measured on MI355X, us: 64 sequences on 8192 shared and up to 512 own tokens, 64/8 heads of
// 128, bf16: both kinds 41, the join 6.6 (everything unshared: 201). The shared tokens alone
// take 10.7 and 1.5 for each 64 of a part's tokens (16 here), which is start and end and the
// matrix units; beside the own tokens' stream 8 more. With two shared workgroups to a unit no
// own ones fit beside them: 65 in all. 128 sequences on 2048 and up to 256, 32/32 heads, fp16,
// are bound by the own tokens' 272 MB: 65 and 5.
//
// In a decode the shared tokens' weights have two 16-bit terms, as all have in the plain call.
// With one, as in the many-token calls, the first case took 43 us instead of 48 and the other
// 67 instead of 70, but the first was 2.3e-3 off 64 bits instead of its outputs' rounding, 1.7e-3.
#include "attn_decode.h"
#include "attn_prefill.h"

namespace qg {
namespace {

template <class F, class PF, bool FP8, int DP, int DU, bool EXACT, bool ONE>
__global__ void __launch_bounds__(256, DP <= 128 ? 2 : 1) attn_parts(SharedArgs p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int block = blockIdx.x + p.first_block;
  if (block < p.shared_blocks) prefill_body<F, PF, FP8, DP, DU, EXACT, kShared, ONE>(p, block, lds);
  else if constexpr (ONE)
    decode_body<F, PF, FP8, DP, EXACT, true>(
        p, (block - p.shared_blocks) * kDecodeWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nullptr);
  else
    prefill_body<F, PF, FP8, DP, DU, EXACT, kOwn>(p, block - p.shared_blocks, lds);
}

template <class F, class PF, bool FP8, int DP, int DU, bool ONE>
hipError_t launch_exact(const SharedArgs& a, int64_t tiles, hipStream_t s) {
  constexpr int lds = PrefillLds<DP>::kTotal;
  const int64_t own = ONE ? (tiles * a.splits + kDecodeWaves - 1) / kDecodeWaves : tiles * a.splits;
  return launch_in_runs(a.shared_blocks + own, [&](dim3 grid, uint32_t first) {
    SharedArgs r = a;
    r.first_block = first;
    if (DU == DP && a.head_dim == DP)
      hipLaunchKernelGGL((attn_parts<F, PF, FP8, DP, DP, true, ONE>), grid, dim3(256), lds, s, r);
    else
      hipLaunchKernelGGL((attn_parts<F, PF, FP8, DP, DU, false, ONE>), grid, dim3(256), lds, s, r);
  });
}

template <class F, class PF, bool FP8, bool ONE>
hipError_t launch_dim(const SharedArgs& a, int64_t tiles, hipStream_t s) {
  if (a.head_dim <= 64) return launch_exact<F, PF, FP8, 64, 64, ONE>(a, tiles, s);
  if (a.head_dim <= 96) return launch_exact<F, PF, FP8, 128, 96, ONE>(a, tiles, s);
  if (a.head_dim <= 128) return launch_exact<F, PF, FP8, 128, 128, ONE>(a, tiles, s);
  if (a.head_dim <= 192) return launch_exact<F, PF, FP8, 256, 192, ONE>(a, tiles, s);
  return launch_exact<F, PF, FP8, 256, 256, ONE>(a, tiles, s);
}

template <bool ONE>
hipError_t launch_parts(const SharedArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s) {
  if (bf16) return fp8 ? launch_dim<BF16, F16, true, ONE>(a, tiles, s) : launch_dim<BF16, BF16, false, ONE>(a, tiles, s);
  return fp8 ? launch_dim<F16, F16, true, ONE>(a, tiles, s) : launch_dim<F16, F16, false, ONE>(a, tiles, s);
}

}  // namespace
}  // namespace qg
