// One new token per sequence over shared and own tokens, and the join of both.
#include "attn_shared_parts.h"

namespace qg {
namespace {

// A thread takes four outputs of a head at a time, `chunks` workgroups a sequence: its own
// parts in order, then the shared ones. A launch of its own rather than the last workgroup's
// work: what a sequence's rows need comes from workgroups of both kinds. 64 sequences of 64
// heads, 8 shared parts: 6.5 us for 20 MB of parts from the caches, most of it the launch and
// the chain of length, group and parts.
template <class F>
__global__ void __launch_bounds__(256) attn_join_one(SharedArgs p, int chunks) {
  const uint32_t block = blockIdx.x + p.first_block;
  const int seq = (int)(block / (uint32_t)chunks), chunk = (int)(block - (uint32_t)seq * (uint32_t)chunks);
  const int len = min(max(scalar_load(p.lens + seq), 0), p.max_len);
  const int shared = shared_tokens(p, seq);
  const Visible see(len, p.window ? len - p.window : 0, p.window ? p.sinks : 0);
  const OwnBlocks own = own_blocks(p, see, shared);
  const int quads = p.head_dim / 4, all = p.kv_heads * p.group * quads;
  for (int x = chunk * 256 + threadIdx.x; x < all; x += chunks * 256) {
    const int head = x / quads, d = 4 * (x - head * quads);
    const int kv_head = head / p.group, in_group = head - kv_head * p.group;
    const int64_t tile = ((int64_t)seq * p.kv_heads + kv_head) * p.row_tiles + in_group / kDecodeRows;
    const int64_t first = tile * p.splits * p.part_rows + in_group % kDecodeRows;
    RowSums sums;
    add_parts(sums, own.parts, [&](int s, f32x4& y, float& m, float& l) {
      const int64_t at = first + (int64_t)s * p.part_rows;
      y = *reinterpret_cast<const f32x4*>(p.partial + at * p.head_dim + d);
      const f32x2 ml = *reinterpret_cast<const f32x2*>(p.stats + 2 * at);
      m = ml[0];
      l = ml[1];
    });
    add_shared_parts(sums, p, shared, kv_head, seq * p.group + in_group, d);
    typename F::T* dst = static_cast<typename F::T*>(p.out) + seq * p.o_ts + head * p.o_hs + d;
    *reinterpret_cast<u32x2*>(dst) = finish<F>(sums.o, sums.total, p.v_scale);
  }
}

}  // namespace

hipError_t launch_attn_decode_shared(const SharedArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s) {
  const hipError_t e = launch_parts<true>(a, bf16, fp8, tiles, s);
  if (e != hipSuccess) return e;
  const int chunks = (a.kv_heads * a.group * (a.head_dim / 4) + 255) / 256;
  return launch_in_runs((int64_t)a.num_seqs * chunks, [&](dim3 grid, uint32_t first) {
    SharedArgs r = a;
    r.first_block = first;
    if (bf16) hipLaunchKernelGGL((attn_join_one<BF16>), grid, dim3(256), 0, s, r, chunks);
    else hipLaunchKernelGGL((attn_join_one<F16>), grid, dim3(256), 0, s, r, chunks);
  });
}

}  // namespace qg
