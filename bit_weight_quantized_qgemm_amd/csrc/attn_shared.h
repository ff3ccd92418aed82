// Device-side helpers of attention over tokens that several sequences share: which group
// a sequence or a tile of rows belongs to, and the join of what was computed for both kinds
// of tokens.
#pragma once

#include <type_traits>

#include "attn_device.h"

namespace qg {

// Number of the entries 0..n-1 that are at most x, for entries that never fall; the same in
// all lanes of a wave, which looks at 64 of them at a time (two rounds up to 4096). Whatever
// the entries hold, only those are read and the loop ends: n falls in every turn.
template <class Entry>
__device__ __forceinline__ int count_up_to(int n, int x, const Entry& entry) {
  const int lane = threadIdx.x & 63;
  int first = 0;
  while (n > 0) {
    const int step = (n + 63) / 64, i = lane * step;
    const int below = __popcll(__ballot(i < n && entry(first + min(i, n - 1)) <= x));
    if (step == 1 || below == 0) return first + below;
    const int skip = (below - 1) * step + 1;   // entries known to be at most x
    first += skip;
    n = min(step - 1, n - skip);
  }
  return first;
}

__device__ __forceinline__ int bounded_seq(const SharedArgs& p, int seq) { return min(max(seq, 0), p.num_seqs); }
// Tokens taken as shared of a group that says `len`: whole blocks, so that both parts of a
// context consist of whole ones (the rest is read through each sequence's own entries).
__device__ __forceinline__ int whole_blocks(const SharedArgs& p, int len) {
  return min(max(len, 0), p.max_shared) / kTokBlock * kTokBlock;
}
// First row of q of sequence seq (tokens are sequences in a call with one token each).
__device__ __forceinline__ int token_of(const SharedArgs& p, int seq) {
  return p.q_start ? min(max(p.q_start[seq], 0), p.num_tokens) : seq;
}

// Tiles of 128 rows. Up to 64 groups, one per lane, they are numbered group after group by a
// prefix sum, so that those without rows come last. Beyond, group g, whose first row is number
// r of all, begins with tile r / 128 + g: it needs at most n / 128 + 1 tiles (rounded down) for
// n rows, so the next one's first is past its last.
__device__ __forceinline__ int tiles_before(const SharedArgs& p, int token, int token_end) {
  const int lane = threadIdx.x & 63;
  const int mine = (max(0, token_end - token) * p.group + kPrefillRows - 1) / kPrefillRows;
  int to = lane < p.num_groups ? mine : 0;
  const int own = to;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int x = __shfl_up(to, d, 64);
    if (lane >= d) to += x;
  }
  return to - own;
}

// Tokens that sequence seq shares (0: it is in no group). Up to 64 groups, all that is asked for
// comes in one go.
__device__ __forceinline__ int shared_tokens(const SharedArgs& p, int seq) {
  const int lane = threadIdx.x & 63;
  int n, first, shared;
  if (p.num_groups <= 64) {
    const int at = min(lane, p.num_groups - 1), raw = p.group_start[at], len = p.shared_lens[at];
    const int raw_end = p.group_start[at + 1];
    n = __popcll(__ballot(lane < p.num_groups && raw <= seq));
    if (n < 1 || __builtin_amdgcn_readlane(raw_end, n - 1) <= seq) return 0;
    first = __builtin_amdgcn_readlane(raw, n - 1);
    shared = __builtin_amdgcn_readlane(len, n - 1);
  } else {
    n = count_up_to(p.num_groups + 1, seq, [&](int i) { return p.group_start[i]; });
    if (n < 1 || n > p.num_groups) return 0;
    first = scalar_load(p.group_start + n - 1);
    shared = scalar_load(p.shared_lens + n - 1);
  }
  return first > seq ? 0 : whole_blocks(p, shared);   // entries that fall
}

// The group of a tile of 128 rows.
struct GroupRows {
  int seq;                // first sequence
  int token, token_end;   // rows of q
  int first_tile;
  int shared;
};
__device__ __forceinline__ GroupRows group_of_tile(const SharedArgs& p, int t) {
  const int lane = threadIdx.x & 63;
  GroupRows r{0, 0, 0, 0, 0};
  int n;
  if (p.num_groups <= 64) {
    const int at = min(lane, p.num_groups - 1);
    const int seq = bounded_seq(p, p.group_start[at]), end = bounded_seq(p, p.group_start[at + 1]), len = p.shared_lens[at];
    const int token = token_of(p, seq), token_end = token_of(p, end), first = tiles_before(p, token, token_end);
    // the last group that begins up to t and has rows
    const uint64_t up_to = __ballot(lane < p.num_groups && first <= t && token < token_end);
    if (up_to == 0) return r;
    n = 64 - __builtin_clzll(up_to);
    r.seq = __builtin_amdgcn_readlane(seq, n - 1);
    r.token = __builtin_amdgcn_readlane(token, n - 1);
    r.token_end = __builtin_amdgcn_readlane(token_end, n - 1);
    r.first_tile = __builtin_amdgcn_readlane(first, n - 1);
    r.shared = whole_blocks(p, __builtin_amdgcn_readlane(len, n - 1));
  } else {
    auto first_tile = [&](int g) { return token_of(p, bounded_seq(p, p.group_start[g])) * p.group / kPrefillRows + g; };
    n = count_up_to(p.num_groups, t, first_tile);
    if (n < 1) return r;
    r.seq = __builtin_amdgcn_readfirstlane(bounded_seq(p, p.group_start[n - 1]));
    r.token = __builtin_amdgcn_readfirstlane(token_of(p, r.seq));
    r.token_end = __builtin_amdgcn_readfirstlane(token_of(p, bounded_seq(p, p.group_start[n])));
    r.first_tile = r.token * p.group / kPrefillRows + n - 1;
    r.shared = whole_blocks(p, scalar_load(p.shared_lens + n - 1));
  }
  if (r.seq >= p.num_seqs || r.first_tile > t) r.token_end = r.token;   // entries that fall
  return r;
}

// Position in its own sequence of row `row` of a group whose first row of q is `token` and first
// sequence `seq`; -1 for a row that the call does not compute. Whole waves call it, for rows
// between `first` and `last`.
__device__ __forceinline__ int position_of(const SharedArgs& p, int seq, int token, int row, int first, int last) {
  const int mine = token + divide(row, p.inv_group);
  if (!p.q_start) return min(max(p.lens[mine], 0), p.max_len) - 1;
  const int from = token + divide_uniform(first, p.inv_group), to = token + divide_uniform(last, p.inv_group);
  // the sequence of the first row's token, then those that begin up to the last one's
  int my_seq = seq + count_up_to(p.num_seqs - seq, from, [&](int i) { return p.q_start[seq + 1 + i]; });
  for (int s = __builtin_amdgcn_readfirstlane(my_seq) + 1; s <= p.num_seqs; s += 64) {
    const int starts = p.q_start[min(s + (int)(threadIdx.x & 63), p.num_seqs)], n = min(64, p.num_seqs - s + 1);
    bool more = true;
    for (int i = 0; i < n && more; ++i) {
      const int start = __builtin_amdgcn_readlane(starts, i);
      more = start <= to;
      my_seq += more && start <= mine;
    }
    if (!more) break;
  }
  if (my_seq >= p.num_seqs) return -1;
  const int q0 = token_of(p, my_seq), q1 = token_of(p, my_seq + 1);
  const int rows = min(max(q1 - q0, 0), p.max_q), i = mine - q0;
  const int len = min(max(p.lens[my_seq], 0), p.max_len);
  return i >= 0 && i < rows ? len - rows + i : -1;
}

// A sequence's virtual blocks past the tokens that it shares, in parts of whole steps: up to
// own_parts parts, and where those would be longer than own_part_blocks (more own tokens than
// the plan took the sequences to have) up to `splits`.
struct OwnBlocks {
  int first, split_blocks, parts;
};
__device__ __forceinline__ OwnBlocks own_blocks(const SharedArgs& p, const Visible& see, int shared) {
  const int block = shared / kTokBlock, step = p.split_step;
  OwnBlocks o;
  o.first = block <= see.sink_blocks ? block : max(see.sink_blocks, block - see.skip);
  const int blocks = max(0, see.blocks - o.first);
  const int each = max((blocks + p.splits - 1) / p.splits, min((blocks + p.own_parts - 1) / p.own_parts, p.own_part_blocks));
  o.split_blocks = max(step, (each + step - 1) / step * step);
  o.parts = max(1, (blocks + o.split_blocks - 1) / o.split_blocks);
  return o;
}

// Where a part of a row's sums stands: row token * group + (head in its group) of a key-value head.
// Places of a tile that hold no row (of a group with few, or that max_q allows and no sequence has)
// take no memory, and the rows of a tile stand together (24 x up to 200 tokens on 2048, 32/32
// heads of 80: 116 us, 118 with the heads of a token together).
__device__ __forceinline__ int64_t part_place(const SharedArgs& p, int part, int kv_head, int row) {
  return ((int64_t)part * p.kv_heads + kv_head) * ((int64_t)p.num_tokens * p.group) + row;
}

// Four outputs of a row before the division: reference maximum, sum of weights, sums.
struct RowSums {
  float m = kNegInf, total = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
};
// Adds parts s..s+N-1 to them, in order; load(s, y, m, l) gives the four sums, the maximum and
// the sum of weights of part s.
template <int N, class Load>
__device__ __forceinline__ void add_batch(RowSums& r, int s, const Load& load) {
  f32x4 y[N];
  float ym[N], yl[N];
#pragma unroll
  for (int u = 0; u < N; ++u) load(s + u, y[u], ym[u], yl[u]);
  float top = r.m;
#pragma unroll
  for (int u = 0; u < N; ++u) top = fmaxf(top, ym[u]);
  const float base = top == kNegInf ? 0.f : top;
  const float f0 = exp2_of(r.m - base);
  r.total *= f0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.o[i] *= f0;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const float f = exp2_of(ym[u] - base);
    r.total += f * yl[u];
#pragma unroll
    for (int i = 0; i < 4; ++i) r.o[i] += f * y[u][i];
  }
  r.m = top;
}
// All of `parts` parts, eight in flight together.
template <class Load>
__device__ __forceinline__ void add_parts(RowSums& r, int parts, const Load& load) {
  int s = 0;
  for (; parts - s >= 8; s += 8) add_batch<8>(r, s, load);
  if (parts - s >= 4) add_batch<4>(r, s, load), s += 4;
  if (parts - s >= 2) add_batch<2>(r, s, load), s += 2;
  if (parts - s >= 1) add_batch<1>(r, s, load);
}
// Adds the shared parts of row `row` of a key-value head: values d..d+3.
__device__ __forceinline__ void add_shared_parts(RowSums& r, const SharedArgs& p, int shared, int kv_head, int row,
                                                 int d) {
  const int parts = (shared / kTokBlock + p.shared_split_blocks - 1) / p.shared_split_blocks;
  add_parts(r, parts, [&](int s, f32x4& y, float& m, float& l) {
    const int64_t at = part_place(p, s, kv_head, row);
    y = *reinterpret_cast<const f32x4*>(p.shared_partial + at * p.head_dim + d);
    const f32x2 ml = *reinterpret_cast<const f32x2*>(p.shared_stats + 2 * at);
    m = ml[0];
    l = ml[1];
  });
}

}  // namespace qg
