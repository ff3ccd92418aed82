// Causal attention of several new tokens per sequence over the paged cache.
//
// A workgroup of four waves takes 128 rows of one sequence and key-value head. A
// row is one query head of one new token, the heads of a token side by side, so
// heads that share keys share the workgroup's tiles of K and V. Each wave owns 32
// rows as the columns of 32x32x16 matrix products: scores S^T = K q^T of 32
// tokens at a time, a running maximum and sum per row in registers (fp32), and
// outputs O^T = V^T P^T.
//
// Tiles of K and V (64 tokens of any four 16-token blocks; 32 for heads above 128
// values) go to LDS, three slots of K and two of V, with one barrier per tile: in
// the turn of tile t, V of tile t + 1 and K of tile t + 2 are on their way.
//   K    rows of 16-byte chunks, chunk number xor token, so that the 16 tokens that
//        are read together (one chunk each) lie in different banks.
//   V    rows as in memory; the operand wants 4 consecutive tokens of one dimension
//        per lane, which the transposing LDS read gives: 16 lanes read 4 tokens of
//        16 dimensions. Its 64-byte units are permuted by token so that those 4
//        tokens lie in different banks.
//   P    the scores leave the matrix unit with row c and tokens 8x + 4h .. + 3 in
//        lane (c, h) = (lane % 32, lane / 32): two such runs are the second operand
//        of the next product as they stand, if V's tokens come in the same order.
// The scores of the next 32 tokens are computed beside the exponentials of the
// present ones, so the matrix and vector units of a SIMD work at the same time in
// each of its two waves. The weights P are rounded once to 16 bits for the matrix
// unit, and summed as rounded, so that a row's weights still add up to one: each is off
// by up to 2^-11 (fp16; no finer than 2^-36 of the largest) or 2^-8 (bf16) of itself,
// an output by as much of the sum of weights times |v|, which is about what rounding
// the output costs where the values do not cancel. A second term, as for single
// tokens, took 20.7 us instead of 18.2 for 2 x 5 tokens on 6001. Statistics, sums and
// accumulators stay fp32.
//
// Bound by the matrix unit and, with it, by power: 8192 tokens, 64/8 heads of 128,
// bf16, take 1010 to 1040 us by device (1057 to 1090 TFLOP/s; a library product of
// 8192^3 reaches 1230 to 1250), at 1.95 GHz of 2.4 and with the matrix unit busy in 53 % of the cycles. 64 rows per
// wave took 1058 us on a device where this takes 1026, eight waves per workgroup 1011
// (but 512 tokens on 4096 then take 108 us instead of 77). Other heads, 4096 tokens of
// 32/8: 80 values 118 to 130 us (660 to 730 TFLOP/s), 96 123 to 127, 192 267 to 274;
// 16/8 of 256 161 to 168. A window of 1024 tokens
// leaves 17 turns per workgroup: 162 us for 8192 tokens of 32/8 heads, e4m3, of which
// a workgroup's start and end take 8 of 41 us.
#pragma once

#include "attn_device.h"
#include "attn_shared.h"

namespace qg {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_t;
typedef const __attribute__((address_space(3))) u32x4* lds_u32x4_t;
typedef const __attribute__((address_space(3))) char* lds_char_t;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

// A raw buffer resource as its four words, for the loads below.
__device__ __forceinline__ u32x4 rsrc_words(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, (uint32_t)kRsrcWord3};
}
// 16 bytes per lane straight into LDS, in lane order from byte `dst` on; lanes past
// the resource write zeros. Written out because the compiler waits for every such
// load that it knows of before any LDS read that it cannot tell apart from it (it
// cannot, for the transposing ones), which would undo the prefetch. It has no
// register result; its arrival is waited for by hand (wait_loads). The wait states
// cover M0 and resource words that a lane read has just written.
__device__ __forceinline__ void dma_16(u32x4 r, uint32_t dst, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds"
               :
               : "s"(dst), "s"(r), "v"(voff)
               : "memory", "m0");
}
// Two or four of them, to dst, dst + 1024, ...: the instruction's own offset moves
// both addresses, so load i's voff is 1024 i short.
__device__ __forceinline__ void dma_16_run(u32x4 r, uint32_t dst, const uint32_t (&v)[2]) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\t"
      "buffer_load_dwordx4 %3, %1, 0 offen offset:1024 lds"
      :
      : "s"(dst), "s"(r), "v"(v[0]), "v"(v[1])
      : "memory", "m0");
}
__device__ __forceinline__ void dma_16_run(u32x4 r, uint32_t dst, const uint32_t (&v)[4]) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\t"
      "buffer_load_dwordx4 %3, %1, 0 offen offset:1024 lds\n\t"
      "buffer_load_dwordx4 %4, %1, 0 offen offset:2048 lds\n\t"
      "buffer_load_dwordx4 %5, %1, 0 offen offset:3072 lds"
      :
      : "s"(dst), "s"(r), "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3])
      : "memory", "m0");
}
// At most N vector-memory operations of this wave are still in flight; nothing
// moves across.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  __builtin_amdgcn_sched_barrier(0);
}
// Barrier of the workgroup without a wait for loads in flight; this wave's LDS
// writes are complete.
__device__ __forceinline__ void lds_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0) alone
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

constexpr int kPrefillWaves = 4;

// What a launch computes: attention over the whole context, or one of the two parts of
// it in a batch whose sequences share their first tokens. kShared: the rows of a group
// of sequences on the tokens that they share; kOwn: a sequence's rows on the others.
// Both leave their sums in the workspace, for a join.
enum PrefillMode { kAlone, kShared, kOwn };

template <int DP>
struct PrefillLds {
  static constexpr int kTile = DP <= 128 ? 64 : 32;   // tokens of a tile
  static constexpr int kRow = DP * 2;                  // bytes of a token
  static constexpr int kBytes = kTile * kRow;          // a slot
  static constexpr int kKSlots = 3, kVSlots = 2;
  static constexpr int kV = kKSlots * kBytes;          // the first slot of V
  static constexpr int kTotal = (kKSlots + kVSlots) * kBytes;
  // byte place of 16-byte chunk c of token t
  static __device__ __forceinline__ int k_turn(int t) { return DP == 64 ? (t >> 1) & 7 : t & 15; }
  static __device__ __forceinline__ int v_turn(int t) { return (DP == 64 ? (t >> 1) & 1 : t & 3) << 2; }
  static __device__ __forceinline__ int k_at(int t, int c) { return t * kRow + ((c ^ k_turn(t)) << 4); }
  static __device__ __forceinline__ int v_at(int t, int c) { return t * kRow + ((c ^ v_turn(t)) << 4); }
};

// A row tile: its sequence, rows and what they see.
struct RowTile {
  int seq, kv_head, row0, rows, all_rows;
  int q0;                   // first row of q of the sequence
  int pos0;                 // position of the first new token
  int pos_min, pos_max;
  Visible see;              // what any of its rows sees
  int parts;
  int v_first = 0;          // first virtual block and blocks of a part (kShared, kOwn)
  int split_blocks = 0;
};
// Key-value heads innermost: the workgroups of one head, which read the same
// tiles, land on one XCD where there are 8 of them (or a multiple); the last rows,
// which see most, first.
__device__ __forceinline__ RowTile row_tile_of(const AttnArgs& p, int tile) {
  const int t = divide_uniform(tile, p.inv_kv_heads), kv_head = tile - t * p.kv_heads;
  const int back = p.num_seqs == 1 ? t : divide_uniform(t, p.inv_seqs), seq = t - back * p.num_seqs;
  const int row0 = (p.row_tiles - 1 - back) * kPrefillRows;
  const int len = min(max(scalar_load(p.lens + seq), 0), p.max_len);
  const int q0 = min(max(scalar_load(p.q_start + seq), 0), p.num_tokens);
  const int q1 = min(max(scalar_load(p.q_start + seq + 1), q0), p.num_tokens);
  const int new_tokens = min(q1 - q0, p.max_q);
  const int all_rows = new_tokens * p.group;
  const int rows = min(kPrefillRows, all_rows - row0);   // <= 0: none
  const int pos0 = len - new_tokens;
  const int pos_min = pos0 + divide_uniform(row0, p.inv_group);
  const int pos_max = pos0 + divide_uniform(row0 + max(1, rows) - 1, p.inv_group);
  const Visible see(max(0, pos_max + 1), p.window ? pos_min - p.window + 1 : 0, p.window ? p.sinks : 0);
  const int parts = p.splits == 1 ? 1 : min(p.splits, max(1, (see.blocks + p.split_blocks - 1) / p.split_blocks));
  return RowTile{seq, kv_head, row0, rows, all_rows, q0, pos0, pos_min, pos_max, see, parts};
}
// The same tile without the tokens that its sequence shares.
__device__ __forceinline__ RowTile own_tile_of(const SharedArgs& p, int tile) {
  RowTile rt = row_tile_of(p, tile);
  const OwnBlocks own = own_blocks(p, rt.see, shared_tokens(p, rt.seq));
  rt.v_first = own.first;
  rt.split_blocks = own.split_blocks;
  rt.parts = own.parts;
  return rt;
}
// A row tile of a group: its rows are those of all its sequences' new tokens, which
// stand one after the other in q. Where positions differ, see and pos_* are for the
// caller to fill in.
__device__ __forceinline__ RowTile shared_tile_of(const SharedArgs& p, int t, int kv_head) {
  const GroupRows g = group_of_tile(p, t);
  const int all_rows = (g.token_end - g.token) * p.group;
  const int row0 = max(0, t - g.first_tile) * kPrefillRows;
  const int rows = min(kPrefillRows, all_rows - row0);   // <= 0: none
  const int blocks = g.shared / kTokBlock;
  RowTile rt{g.seq, kv_head, row0, rows, all_rows, g.token, 0, 0, 0, Visible(g.shared, 0, 0),
             (blocks + p.shared_split_blocks - 1) / p.shared_split_blocks};
  rt.split_blocks = p.shared_split_blocks;
  return rt;
}

template <PrefillMode MODE>
using PrefillArgs = std::conditional_t<MODE == kAlone, AttnArgs, SharedArgs>;

// DP: values of a head's place in LDS; DU: those that take part in the products. block:
// workgroup among those of this kind. TWO: the weights go in as two 16-bit terms and are
// summed unrounded, as in attn_decode.h.
template <class F, class PF, bool FP8, int DP, int DU, bool EXACT, PrefillMode MODE, bool TWO = false>
__device__ __forceinline__ void prefill_body(const PrefillArgs<MODE>& p, int block, char* lds) {
  using L = PrefillLds<DP>;
  using T = typename F::T;
  constexpr int kElt = FP8 ? 1 : 2;
  constexpr int kBlocks = L::kTile / kTokBlock;       // blocks of a tile
  constexpr int kHalves = L::kTile / 32;              // steps of a tile
  constexpr int kMine = L::kTile / kPrefillWaves;     // tokens of a tile that a wave loads
  constexpr int kLanes = DP * kElt / 16;              // lanes that load one token
  constexpr int kRows = 64 / kLanes;                  // tokens of a load
  constexpr int kLoads = kMine / kRows;
  constexpr int kSteps = DU / 16;
  constexpr int kDB = DU / 32;

  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int split, tile;
  if constexpr (MODE == kShared) {
    // key-value heads innermost, and rows outermost: tiles without rows come last
    const int x = divide_uniform(block, p.inv_kv_heads), t = divide_uniform(x, p.inv_shared_splits);
    split = x - t * p.shared_splits, tile = t * p.kv_heads + block - x * p.kv_heads;
  } else {
    const int tiles = p.num_seqs * p.kv_heads * p.row_tiles;
    split = p.splits == 1 ? 0 : divide_uniform(block, p.inv_tiles), tile = block - split * tiles;
  }
  RowTile rt = [&]() {
    if constexpr (MODE == kAlone) return row_tile_of(p, tile);
    else if constexpr (MODE == kOwn) return own_tile_of(p, tile);
    else return shared_tile_of(p, tile / p.kv_heads, tile % p.kv_heads);
  }();
  if (rt.rows <= 0 || split >= rt.parts) return;

  // ---- kShared: positions of this lane's row and of the wave's
  constexpr int kFar = INT32_MAX / 2;   // past every position
  int shared_pos = -1, shared_min = kFar, shared_max = -1;
  if constexpr (MODE == kShared) {
    const int first = rt.row0 + wave * 32, r = first + c, end = rt.row0 + rt.rows;
    if (first < end)
      shared_pos = position_of(p, rt.seq, rt.q0, min(r, end - 1), first, min(first + 31, end - 1));
    if (r >= end) shared_pos = -1;
    shared_min = r < end ? shared_pos : kFar;
    shared_max = shared_pos;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      shared_min = min(shared_min, __shfl_xor(shared_min, d, 64));
      shared_max = max(shared_max, __shfl_xor(shared_max, d, 64));
    }
    shared_min = __builtin_amdgcn_readfirstlane(shared_min);
    shared_max = __builtin_amdgcn_readfirstlane(shared_max);
    if (p.window) {   // the first token that any of the tile's rows has in its window
      int32_t* least = reinterpret_cast<int32_t*>(lds);
      if (lane == 0) least[wave] = shared_min;
      lds_barrier();
      const int tile_min = min(min(least[0], least[1]), min(least[2], least[3]));
      const int low = max(0, __builtin_amdgcn_readfirstlane(tile_min) - p.window + 1);
      rt.see = Visible(rt.see.len, min(low, rt.see.len), p.sinks);
      lds_barrier();
    }
  }
  const Visible& see = rt.see;
  const int split_blocks = MODE == kAlone ? p.split_blocks : rt.split_blocks;
  const int v_begin = rt.v_first + split * split_blocks, v_end = min(see.blocks, v_begin + split_blocks);
  const int turns = (v_end - v_begin + kBlocks - 1) / kBlocks;   // tiles

  // ---- this lane's row, and the wave's span of positions
  const int row = rt.row0 + wave * 32 + c;
  const bool live = row < rt.all_rows;
  const int qi = live ? divide(row, p.inv_group) : 0;
  const int head = rt.kv_head * p.group + (live ? row - qi * p.group : 0);
  const int pos = MODE == kShared ? shared_pos : live ? rt.pos0 + qi : -1;
  const int low = p.window ? pos - p.window + 1 : 0;
  const int wave_rows = min(32, rt.rows - wave * 32);   // may be <= 0
  const int wave_min = MODE == kShared ? shared_min : rt.pos0 + divide_uniform(rt.row0 + wave * 32, p.inv_group);
  const int wave_max =
      MODE == kShared ? shared_max
      : wave_rows > 0 ? rt.pos0 + divide_uniform(rt.row0 + wave * 32 + wave_rows - 1, p.inv_group) : -1;
  const int wave_low = p.window ? wave_max - p.window + 1 : 0;   // every row of the wave sees low..min

  u32x4 q[kSteps];
  auto load_q = [&]() {
    const T* src = static_cast<const T*>(p.q) + (int64_t)(rt.q0 + qi) * p.q_ts + head * p.q_hs;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = 16 * s + 8 * h;
      q[s] = u32x4{0, 0, 0, 0};
      if (live && d < p.head_dim) q[s] = *reinterpret_cast<const u32x4*>(src + d);
    }
  };

  // ---- pages
  const int32_t* table = p.cache.table + rt.seq * p.cache.table_stride;
  auto entry_at = [&](int v) {   // table entry of virtual block v; -1 past the end
    int place;
    const int col = page_of(p.cache, v < v_end ? see.block(v) : 0, &place);
    return v < v_end ? table[col] : -1;
  };
  auto page_in = [&](int entry) { return entry < p.cache.num_pages ? entry : -1; };
  // ---- loads: this wave's tokens of a tile, all of one block
  const int my_block = wave * kMine / kTokBlock, my_first = wave * kMine % kTokBlock;
  const uint32_t ts_bytes = (uint32_t)p.cache.token_stride * kElt;
  const char* kbase = static_cast<const char*>(p.cache.k) + rt.kv_head * p.cache.head_stride * kElt;
  const char* vbase = static_cast<const char*>(p.cache.v) + rt.kv_head * p.cache.head_stride * kElt;
  const int l_row = lane / kLanes, l_place = lane % kLanes;
  // 16-bit caches go straight to LDS, 16 bytes per lane in lane order: the lane at
  // a permuted place fetches the chunk that belongs there. e4m3 caches go through
  // registers, in memory order.
  uint32_t koff[kLoads], voff[kLoads];   // of each load, within the block
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int t = my_first + i * kRows + l_row;
    auto off = [&](int chunk) { return EXACT || chunk * 16 < p.head_dim * kElt ? t * ts_bytes + chunk * 16 : 0x80000000u; };
    koff[i] = off(FP8 ? l_place : l_place ^ L::k_turn(wave * kMine + i * kRows + l_row));
    voff[i] = off(FP8 ? l_place : l_place ^ L::v_turn(i * kRows + l_row));
    // the tokens of a whole head cover at least 1024 i bytes
    if (EXACT && !FP8) {
      koff[i] -= i * 1024;
      voff[i] -= i * 1024;
    }
  }
  u32x4 kr[FP8 ? kLoads : 1], vr[FP8 ? kLoads : 1];
  // Where 64 consecutive blocks lie, one per lane (no bytes where there is no page):
  // the present group of tiles; the table entries of the next are fetched half a
  // group early. Where a page is out of range, the masks of that group's tiles, and
  // of those before it that are still in use, have to look.
  constexpr int kGroup = 64 / kBlocks;
  uint32_t at_low = 0, at_high = 0, at_bytes = 0;
  int next_entries = -1;
  bool missing = false, look = false;
  auto enter = [&](int turn, int entries) {
    const int v = v_begin + turn * kBlocks + lane, page = page_in(entries), blk = v < v_end ? see.block(v) : 0;
    int place;
    page_of(p.cache, blk, &place);
    const int64_t at = (page * p.cache.page_stride + (int64_t)place * kTokBlock * p.cache.token_stride) * kElt;
    at_low = (uint32_t)at;
    at_high = (uint32_t)(at >> 32);
    at_bytes = page < 0 ? 0u : min(kTokBlock, see.len - blk * kTokBlock) * ts_bytes;
    const bool before = missing;
    missing = __any(page < 0 && v < v_end);
    look = missing || before;
  };
  // this wave's block of a tile
  struct Where {
    uint64_t at;
    uint32_t bytes;
  };
  auto find = [&](int turn) {
    const int x = (turn % kGroup) * kBlocks + my_block;
    Where w;
    w.at = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_low, x) |
           (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_high, x) << 32;
    w.bytes = __builtin_amdgcn_readlane(at_bytes, x);
    return w;
  };
  const uint32_t lds_mine =
      __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_ptr_t)lds) + wave * kMine * L::kRow;
  auto issue = [&](const char* base, const Where& w, int slot, const uint32_t (&off)[kLoads],
                   u32x4 (&regs)[FP8 ? kLoads : 1]) {   // slot: byte offset in LDS
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) regs[i] = load16(make_rsrc(base + w.at, w.bytes), off[i], 0);
    } else {
      const u32x4 r = rsrc_words(base + w.at, w.bytes);
      if constexpr (EXACT) {
        dma_16_run(r, lds_mine + slot, off);
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) dma_16(r, lds_mine + slot + i * 1024, off[i]);
      }
    }
  };
  auto issue_k = [&](const Where& w, int slot) { issue(kbase, w, slot, koff, kr); };
  auto issue_v = [&](const Where& w, int slot) { issue(vbase, w, slot, voff, vr); };
  // e4m3: widens what was loaded and writes it to its slot
  auto widen_k = [&](int slot) {
#pragma unroll
    for (int i = 0; i < (FP8 ? kLoads : 0); ++i) {
      const int t = wave * kMine + i * kRows + l_row;
      u32x4 k[2];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        k[w / 2][2 * (w % 2)] = F::template from_fp8<false>(kr[i][w]);
        k[w / 2][2 * (w % 2) + 1] = F::template from_fp8<true>(kr[i][w]);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) *reinterpret_cast<u32x4*>(lds + slot + L::k_at(t, 2 * l_place + w)) = k[w];
    }
  };
  auto widen_v = [&](int slot) {
#pragma unroll
    for (int i = 0; i < (FP8 ? kLoads : 0); ++i) {
      const int t = wave * kMine + i * kRows + l_row;
      u32x4 v[2];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[w / 2][2 * (w % 2)] = PF::template from_fp8<false>(vr[i][w]);
        v[w / 2][2 * (w % 2) + 1] = PF::template from_fp8<true>(vr[i][w]);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) *reinterpret_cast<u32x4*>(lds + slot + L::v_at(t, 2 * l_place + w)) = v[w];
    }
  };
  // Values that no row of the tile sees, in a block that is partly seen (the first
  // of the window, the last with sinks), are zeroed in LDS: the turns of this
  // wave's blocks of that kind, or -1.
  auto turn_of = [&](int v, bool there) {
    const int x = v - v_begin;
    return there && x >= 0 && v < v_end && x % kBlocks == my_block ? x / kBlocks : -1;
  };
  const int cut_low = turn_of(see.low / kTokBlock - see.skip, see.low % kTokBlock != 0);
  const int cut_sink = turn_of(see.sinks / kTokBlock, see.sinks % kTokBlock != 0);
  auto cut = [&](int turn, int slot) {
    const int j0 = see.block(v_begin + turn * kBlocks + my_block) * kTokBlock;
    constexpr int kChunks = DP / 8;
    for (int x = lane; x < kMine * kChunks; x += 64)
      if (!see.sees(j0 + my_first + x / kChunks))
        *reinterpret_cast<u32x4*>(lds + slot + wave * kMine * L::kRow + x * 16) = u32x4{0, 0, 0, 0};
  };

  float mref = kNegInf, sum = 0.f;
  f32x16 acc[kDB];
#pragma unroll
  for (int d = 0; d < kDB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;

  // ---- operand addresses, in the slots of the present tile
  lds_char_t ka[kSteps], va[kDB];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) ka[k] = (lds_char_t)lds + L::k_at(c, 2 * k + h);
  // transposing read: the lane reads 8 bytes of token (lane % 16) / 4 of its run of
  // four, dimensions 16 * (lane / 16 % 2) + 4 * (lane % 4)
#pragma unroll
  for (int d = 0; d < kDB; ++d)
    va[d] = (lds_char_t)lds + L::kV + L::v_at(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) + (lane & 1) * 8;

  // scores of 32 tokens, from their K operands
  auto keys = [&](int half, u32x4 (&k)[kSteps]) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) k[i] = *(lds_u32x4_t)(ka[i] + half * 32 * L::kRow);
  };
  auto scores = [&](const u32x4 (&k)[kSteps]) {
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) s = F::mfma32(k[i], q[i], s);
    return s;
  };
  // steps (32 tokens) of which every row of the wave sees every token
  const int seen_low = p.window ? (max(0, wave_low) + kTokBlock - 1) / kTokBlock - see.skip - v_begin : 0;
  const int seen_high = max(0, wave_min + 1) / kTokBlock - see.skip - v_begin;
  const int whole_first = (max(0, seen_low) + 1) / 2;
  const uint32_t whole_steps = (uint32_t)max(0, max(0, min(seen_high, v_end - v_begin)) / 2 - whole_first);
  // masks the scores of step n, where a row does not see them all
  auto mask = [&](f32x16& s, int n) {
    if (__builtin_expect(!look && (uint32_t)(n - whole_first) < whole_steps, 1)) return;
    const int v0 = v_begin + 2 * n;
    int j0[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      j0[b] = v0 + b < v_end ? see.block(v0 + b) * kTokBlock : INT32_MAX - kTokBlock;
      if (look && page_in(entry_at(v0 + b)) < 0) j0[b] = INT32_MAX - kTokBlock;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int j = j0[i / 8] + 8 * (i / 4 % 2) + 4 * h + i % 4;   // registers 0-7: the first block
      const bool hidden = (j > pos) | ((j < low) & (j >= p.sinks));
      s[i] = hidden ? kNegInf : s[i];
    }
  };
  auto largest = [&](const f32x16& s) {
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    return top * p.scale_log2;
  };
  auto raise = [&](float top) {   // moves the reference maxima, if scores pass them
    if (__builtin_expect(__any(top > raise_limit<PF>(mref)), 0)) {
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float m = fmaxf(mref, top);
      const float f = m == kNegInf ? 1.f : exp2_of(mref - m);
      mref = m;
      sum *= f;
#pragma unroll
      for (int d = 0; d < kDB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] *= f;
    }
  };
  // weights of 16 tokens (u = 0, 1 of a step's 32) as an operand
  u32x4 w[2], rest[2];
  auto weigh = [&](const f32x16& s, int u) {
    const float base = weight_base<PF>(mref);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e0 = exp2_of(__builtin_fmaf(s[8 * u + 2 * i], p.scale_log2, -base));
      const float e1 = exp2_of(__builtin_fmaf(s[8 * u + 2 * i + 1], p.scale_log2, -base));
      const uint32_t x = PF::pack(e0, e1);
      if constexpr (TWO) {
        sum += e0 + e1;
        rest[u][i] = PF::pack(e0 - PF::lo(x), e1 - PF::hi(x));
      } else {
        sum = PF::add_pair(x, sum);
      }
      w[u][i] = x;
    }
  };
  // V operand of dimensions 32 d .., tokens 16 u .. of a half
  auto value = [&](int half, int u, int d) {
    u32x4 v;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const s16x4 r =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(va[d] + (half * 32 + 16 * u + 8 * x) * L::kRow));
      const u32x2 y = __builtin_bit_cast(u32x2, r);
      v[2 * x] = y[0];
      v[2 * x + 1] = y[1];
    }
    return v;
  };
  // One step: scores of the next 32 tokens beside the weights of the first 16 of the
  // present ones, then the outputs of those beside the weights of the other 16, so
  // that vector operations stand between matrix products throughout.
  auto step = [&](int half, int next_half, f32x16& present, f32x16& next, int number, bool more) {
    u32x4 k[kSteps], v[2][kDB];
    __builtin_amdgcn_sched_barrier(0);
    keys(next_half, k);
    __builtin_amdgcn_sched_barrier(0);
    next = scores(k);
    weigh(present, 0);
#pragma unroll
    for (int d = 0; d < kDB; ++d) v[0][d] = value(half, 0, d);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x002, 24 / kSteps, 0);   // vector operations
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);             // a matrix product
      if (i >= kSteps / 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // LDS reads
    }
    asm volatile("" : "+v"(w[0]));   // not moved past the masks
    if constexpr (TWO) asm volatile("" : "+v"(rest[0]));
    __builtin_amdgcn_sched_barrier(0);
    if (more) mask(next, number + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < kDB; ++d) v[1][d] = value(half, 1, d);
    __builtin_amdgcn_sched_barrier(0);
    weigh(present, 1);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int d = 0; d < kDB; ++d) {
        acc[d] = PF::mfma32(v[u][d], w[u], acc[d]);
        if constexpr (TWO) acc[d] = PF::mfma32(v[u][d], rest[u], acc[d]);
      }
    const float top = largest(next);
#pragma unroll
    for (int d = 0; d < kDB; ++d) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 24 / kDB, 0);
    }
#pragma unroll
    for (int d = 0; d < kDB; ++d) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 8 / kDB, 0);
    }
    if (more) raise(top);
  };

  // tiles that some row of the wave sees
  const int wave_blocks = wave_max < 0 ? 0 : min(see.blocks, Visible(wave_max + 1, see.low, see.sinks).blocks);
  const int mine = max(0, min(turns, (wave_blocks - v_begin + kBlocks - 1) / kBlocks));

  // ---- the line of tiles. In the turn of tile t, V of t and K of t + 1 have landed
  // behind the barrier; V of t + 1 and K of t + 2 go to the slots that V and K of
  // t - 1 have left.
  f32x16 s0, s1;
  Where ahead;                  // of tile t + 1
  int kslot = 0, vslot = L::kV;   // of tile t
  auto next_k = [&](int slot) { return slot == (L::kKSlots - 1) * L::kBytes ? 0 : slot + L::kBytes; };
  auto next_v = [&](int slot) { return slot == L::kV + (L::kVSlots - 1) * L::kBytes ? L::kV : slot + L::kBytes; };
  if (turns > 0) {
    const int entries = entry_at(v_begin + lane);
    load_q();   // while the entries are on their way
    enter(0, entries);
    ahead = find(0);
    issue_k(ahead, 0);
    if constexpr (FP8) widen_k(0);
    issue_v(ahead, L::kV);
    ahead = find(1);
    issue_k(ahead, L::kBytes);
    if constexpr (!FP8) wait_loads<0>();
    lds_barrier();
    u32x4 k[kSteps];
    keys(0, k);
    s0 = scores(k);
    mask(s0, 0);
    raise(largest(s0));
  }
  for (int t = 0; t < turns; ++t) {
    const int kslot1 = next_k(kslot);
    if constexpr (FP8) {
      widen_v(vslot);
      widen_k(kslot1);
    } else {
      wait_loads<0>();
    }
    if (__builtin_expect(t == cut_low || t == cut_sink, 0)) cut(t, vslot);
    lds_barrier();
    const int far = t + 2;
    if (__builtin_expect(far % kGroup == 0, 0)) enter(far, next_entries);
    const Where later = find(far);
    if (__builtin_expect(far % kGroup == kGroup / 2, 0)) next_entries = entry_at(v_begin + (far + kGroup / 2) * kBlocks + lane);
    issue_v(ahead, next_v(vslot));
    issue_k(later, next_k(kslot1));
    ahead = later;
    if (t < mine) {
      if constexpr (kHalves == 2) step(0, 1, s0, s1, 2 * t, true);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) ka[k] += kslot1 - kslot;
      if constexpr (kHalves == 2) {
        step(1, 0, s1, s0, 2 * t + 1, t + 1 < mine);
      } else {
        step(0, 0, s0, s1, t, t + 1 < mine);
        s0 = s1;
      }
#pragma unroll
      for (int d = 0; d < kDB; ++d) va[d] += next_v(vslot) - vslot;
    }
    kslot = kslot1;
    vslot = next_v(vslot);
  }
  wait_loads<0>();   // nothing lands in LDS after this workgroup

  // ---- outputs of the wave's rows, or their part
  sum += __shfl_xor(sum, 32, 64);
  if (!live) return;   // both lanes of a row
  if (MODE == kAlone && rt.parts == 1) {
    T* dst = static_cast<T*>(p.out) + (int64_t)(rt.q0 + qi) * p.o_ts + head * p.o_hs;
    const float f = sum == 0.f ? 0.f : p.v_scale / sum;   // zeros where nothing was visible
#pragma unroll
    for (int d = 0; d < kDB; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        // a lane holds dimensions 4 h .. of two runs of eight; after the exchange
        // with its partner, all eight of run h
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const u32x2 x = __builtin_bit_cast(
              u32x2, __builtin_amdgcn_permlane32_swap(F::pack(acc[d][i + 2 * j] * f, acc[d][i + 2 * j + 1] * f),
                                                      F::pack(acc[d][i + 4 + 2 * j] * f, acc[d][i + 5 + 2 * j] * f),
                                                      false, false));
          o[j] = x[0];
          o[2 + j] = x[1];
        }
        const int at = 32 * d + 2 * i + 8 * h;
        if (EXACT || at < p.head_dim) *reinterpret_cast<u32x4*>(dst + at) = o;
      }
    return;
  }
  int64_t r;
  float *partial = p.partial, *stats = p.stats;
  if constexpr (MODE == kAlone) r = ((int64_t)tile * p.splits + split) * p.part_rows + row - rt.row0;
  else r = part_place(p, split, rt.kv_head, rt.q0 * p.group + row);
  if constexpr (MODE == kShared) {
    partial = p.shared_partial;
    stats = p.shared_stats;
  }
  float* dst = partial + r * p.head_dim;
#pragma unroll
  for (int d = 0; d < kDB; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int at = 32 * d + 2 * i + 4 * h;
      if (EXACT || at < p.head_dim)
        *reinterpret_cast<f32x4*>(dst + at) = f32x4{acc[d][i], acc[d][i + 1], acc[d][i + 2], acc[d][i + 3]};
    }
  if (h == 0) *reinterpret_cast<f32x2*>(stats + 2 * r) = f32x2{mref, sum};
}

// Two workgroups of a CU where the heads fit 128 values (two waves per SIMD); the
// accumulators of longer heads take all registers of one wave per SIMD.
template <class F, class PF, bool FP8, int DP, int DU, bool EXACT>
__global__ void __launch_bounds__(256, DP <= 128 ? 2 : 1) attn_prefill(AttnArgs p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  prefill_body<F, PF, FP8, DP, DU, EXACT, kAlone>(p, blockIdx.x + p.first_block, lds);
}

}  // namespace
}  // namespace qg
