// Attention of one new token per sequence over the paged cache.
//
// A workgroup takes one part of one sequence's cached tokens for up to 16 query
// heads of one key-value head: scores S^T = K q^T and outputs O^T = V^T P^T on
// 16x16x32 matrix instructions, with the query heads as columns and the running
// maximum and sum of each head's softmax kept in registers (fp32). Its four waves
// take pairs of 16-token blocks in turn, each with accumulators of its own, and
// meet once at the end; parts meet in the last workgroup to arrive.
//
// Every byte of K and V is used once, so the kernel is bound by the cache's
// stream: 256 contexts of 8192 tokens, 8 heads of 128, bf16, take 1220 to 1330 us by
// device (6.5 to 7.0 TB/s; a bare streaming read of 2 GiB, which has less to spread its
// start and end over, reaches 6.2, a copy 4.9 read and written), one of 131072 in e4m3
// 46 us (5.8 TB/s), 32 of up to 4096 60 us (4.5 TB/s; parts of uneven length). Short contexts are bound by the chain of launch, length, table
// entry, load, join: 1 x 1000 tokens 9.7 us in parts, 12 x 256 7.8 us in one. Loads go
// straight to registers in operand form; through LDS they would cost a barrier per
// pair and bring no reuse:
//   K    lane (c, h) = (lane % 16, lane / 16) loads 16 bytes of token c, which
//        are the first operand's 8 values of one 32-value step (e4m3: of two).
//   V    the operand wants 8 tokens of one dimension per lane, memory has the
//        dimensions of one token together. Lane (c, h) loads the dimensions
//        8c..8c+7 of its 8 tokens (a whole token row per 16 lanes) and picks
//        dimension 8c + i of all 8 with byte permutes: matrix product i of 8
//        then covers the dimensions 8c + i, c = 0..15.
//   P    the scores leave the matrix unit with head c and tokens 4h..4h+3 of
//        each block in lane (c, h): with the tokens of V in that order they are
//        the second operand as they stand. Weights go in as two 16-bit terms (the
//        rounded weight and the rest), good to 2^-22 (fp16) or 2^-16 (bf16) of each
//        and, in fp16, no finer than 2^-36 of the largest; the matrix unit has the
//        time.
// K of the next pair is requested as soon as this pair's scores are done and V
// once its outputs are, so one of the two is always on its way. Tokens past the
// end, pages out of range and dimensions past head_dim are cut off by the size
// of the buffer resource: such loads give zeros and move nothing.
#pragma once

#include "attn_device.h"
#include "attn_shared.h"

namespace qg {
namespace {

template <class F, bool FP8, int DP>
struct DecodeShape {
  static constexpr int kElt = FP8 ? 1 : 2;
  static constexpr int kKLoads = DP * kElt / 64;        // 16-byte loads of K per lane and block
  static constexpr int kSteps = DP / 32;                // 32-value steps of a score
  static constexpr int kVDims = DP >= 128 ? 8 : DP / 16;   // dimensions of a V load
  static constexpr int kVCols = DP / (16 * kVDims);     // V loads per token
  static constexpr int kVWords = kVDims * kElt / 4;
};

// A pair of token blocks: where its two blocks lie.
struct PairAt {
  int blk[2];          // token blocks (-1: absent)
  int64_t at[2];       // element offset of the block's first token
  int rows[2];         // tokens that may be read
};

template <int DP>
struct DecodeLds {
  static constexpr int kOutStride = DP + 4;
  float part[kDecodeWaves][kDecodeRows][kOutStride];
  float part_max[kDecodeWaves][kDecodeRows], part_sum[kDecodeWaves][kDecodeRows];
  int flag;
};

// EXACT: head_dim is DP, so that the loads' offsets need no bounds of their own. OWN: the
// sequence's tokens past those that it shares with others, a wave for each part; the sums stay
// in the workspace, for the join with the shared ones'. block: workgroup (OWN: wave) among
// those of this kind.
template <class F, class PF, bool FP8, int DP, bool EXACT, bool OWN>
__device__ __forceinline__ void decode_body(const std::conditional_t<OWN, SharedArgs, AttnArgs>& p, int block,
                                            DecodeLds<DP>* lds) {
  using S = DecodeShape<F, FP8, DP>;
  using T = typename F::T;
  constexpr int kTurn = OWN ? 1 : kDecodeWaves;   // waves that take pairs in turn
  const int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // all first parts, then all second ones: the parts that a shorter sequence does
  // not have come last, and workgroups 8 apart, which share an XCD, hold every
  // part number in equal shares
  const int heads = p.kv_heads * p.row_tiles;
  const int tiles = p.num_seqs * heads;
  if (OWN && block >= tiles * p.splits) return;
  const int split = p.splits == 1 ? 0 : divide_uniform(block, p.inv_tiles), tile = block - split * tiles;
  const int seq = divide_uniform(tile, p.inv_heads);
  const int row_tile = p.row_tiles == 1 ? 0 : (tile - seq * heads) % p.row_tiles;
  const int kv_head = p.row_tiles == 1 ? tile - seq * heads : (tile - seq * heads) / p.row_tiles;
  const int head0 = kv_head * p.group + row_tile * kDecodeRows;
  const int rows = min(kDecodeRows, p.group - row_tile * kDecodeRows);

  const int len = min(max(scalar_load(p.lens + seq), 0), p.max_len);
  const Visible see(len, p.window ? len - p.window : 0, p.window ? p.sinks : 0);
  // never more than the workspace holds (the plan covers see.blocks with p.splits)
  int parts, split_blocks, v_first = 0;
  if constexpr (OWN) {
    const OwnBlocks own = own_blocks(p, see, shared_tokens(p, seq));
    parts = own.parts;
    split_blocks = own.split_blocks;
    v_first = own.first;
  } else {
    parts = p.splits == 1 ? 1 : min(p.splits, max(1, (see.blocks + p.split_blocks - 1) / p.split_blocks));
    split_blocks = p.split_blocks;
  }
  if (split >= parts) return;
  const int v_end = min(see.blocks, v_first + (split + 1) * split_blocks);

  const int32_t* table = p.cache.table + seq * p.cache.table_stride;
  const uint32_t ts_bytes = (uint32_t)p.cache.token_stride * S::kElt;
  const char* kbase = static_cast<const char*>(p.cache.k) + kv_head * p.cache.head_stride * S::kElt;
  const char* vbase = static_cast<const char*>(p.cache.v) + kv_head * p.cache.head_stride * S::kElt;

  // ---- q as the second operand: column c, 8 values of each 32-value step
  u32x4 q[S::kSteps];
  {
    const T* src = static_cast<const T*>(p.q) + seq * p.q_ts + (head0 + c) * p.q_hs;
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      const int d = FP8 ? 64 * (s / 2) + 16 * h + 8 * (s % 2) : 32 * s + 8 * h;
      q[s] = u32x4{0, 0, 0, 0};
      if (c < rows && d < p.head_dim) q[s] = *reinterpret_cast<const u32x4*>(src + d);
    }
  }

  // ---- loads of a pair of blocks
  const uint32_t kOut = 0x80000000u;   // an offset past any resource
  uint32_t koff[EXACT ? 1 : S::kKLoads];
  if (EXACT) {
    koff[0] = c * ts_bytes + 16 * h;
  } else {
#pragma unroll
    for (int s = 0; s < S::kKLoads; ++s)
      koff[s] = 64 * s + 16 * h < p.head_dim * S::kElt ? c * ts_bytes + 64 * s + 16 * h : kOut;
  }
  uint32_t voff[S::kVCols];
#pragma unroll
  for (int j = 0; j < S::kVCols; ++j) {
    const int d = j * 16 * S::kVDims + c * S::kVDims;
    voff[j] = d < p.head_dim ? 4 * h * ts_bytes + d * S::kElt : kOut;
  }
  u32x4 kr[2][S::kKLoads];
  uint32_t vr[2][4][S::kVCols][S::kVWords];

  auto locate = [&](int pair) {
    PairAt a;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int v = v_first + 2 * pair + s;
      const bool there = v < v_end;
      const int blk = there ? see.block(v) : 0;
      int place;
      const int col = page_of(p.cache, blk, &place);
      const int page = there ? scalar_load(table + col) : -1;
      const bool ok = page >= 0 && page < p.cache.num_pages;
      a.blk[s] = ok ? blk : -1;
      a.rows[s] = ok ? min(kTokBlock, len - blk * kTokBlock) : 0;
      a.at[s] = ok ? page * p.cache.page_stride + (int64_t)place * kTokBlock * p.cache.token_stride : 0;
    }
    return a;
  };
  auto load_k = [&](const PairAt& a) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const rsrc_t r = make_rsrc(kbase + a.at[s] * S::kElt, a.rows[s] * ts_bytes);
#pragma unroll
      for (int i = 0; i < S::kKLoads; ++i)
        kr[s][i] = EXACT ? load16_stream(r, koff[0] + 64 * i, 0) : load16_stream(r, koff[i], 0);
    }
  };
  auto load_v = [&](const PairAt& a) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const rsrc_t r = make_rsrc(vbase + a.at[s] * S::kElt, a.rows[s] * ts_bytes);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < S::kVCols; ++j) {
          if constexpr (S::kVWords == 4) {
            const u32x4 w = load16_stream(r, voff[j], e * ts_bytes);
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[s][e][j][i] = w[i];
          } else if constexpr (S::kVWords == 2) {
            const u32x2 w = load8_stream(r, voff[j], e * ts_bytes);
            vr[s][e][j][0] = w[0];
            vr[s][e][j][1] = w[1];
          } else {
            vr[s][e][j][0] = __builtin_amdgcn_raw_buffer_load_b32(r, voff[j], e * ts_bytes, kStreamPolicy);
          }
        }
    }
  };

  float mref = kNegInf;   // reference maximum of head c (log2 units), same in the lanes of a head
  float sum = 0.f;        // this lane's part of the sum of weights
  f32x4 acc[S::kVCols][S::kVDims];
#pragma unroll
  for (int j = 0; j < S::kVCols; ++j)
#pragma unroll
    for (int i = 0; i < S::kVDims; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int pair_end = (v_end - v_first + 1) / 2;
  int pair = split * split_blocks / 2 + (OWN ? 0 : wave);
  PairAt now = locate(pair);
  load_k(now);
  load_v(now);
  PairAt next = locate(pair + kTurn);
  for (; pair < pair_end; pair += kTurn) {
    // ---- scores of the pair: lane (c, h) gets head c, tokens 4h..4h+3 of each block
    f32x4 sc[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      sc[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < S::kSteps; ++t) {
        u32x4 k;
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = kr[s][t / 2][2 * (t % 2) + i];
            k[2 * i] = F::template from_fp8<false>(w);
            k[2 * i + 1] = F::template from_fp8<true>(w);
          }
        } else {
          k = kr[s][t];
        }
        sc[s] = F::mfma16(k, q[t], sc[s]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_k(next);
    __builtin_amdgcn_sched_barrier(0);

    // ---- softmax weights
    float t[8];
    bool whole = true;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      whole = whole && now.blk[s] >= 0 && see.whole(now.blk[s]);
#pragma unroll
      for (int r = 0; r < 4; ++r) t[4 * s + r] = sc[s][r] * p.scale_log2;
    }
    if (!whole) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (now.blk[s] < 0 || !see.sees(now.blk[s] * kTokBlock + 4 * h + r)) t[4 * s + r] = kNegInf;
    }
    float top = t[0];
#pragma unroll
    for (int r = 1; r < 8; ++r) top = fmaxf(top, t[r]);
    if (__any(top > raise_limit<PF>(mref))) {
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float m = fmaxf(mref, top);
      const float f = m == kNegInf ? 1.f : exp2_of(mref - m);
      mref = m;
      sum *= f;
#pragma unroll
      for (int j = 0; j < S::kVCols; ++j)
#pragma unroll
        for (int i = 0; i < S::kVDims; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[j][i][r] *= f;
    }
    const float base = weight_base<PF>(mref);
    u32x4 w, wl;   // the weights in 16 bits, and what that leaves
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      t[r] = exp2_of(t[r] - base);
      sum += t[r];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      w[r] = PF::pack(t[2 * r], t[2 * r + 1]);
      wl[r] = PF::pack(t[2 * r] - PF::lo(w[r]), t[2 * r + 1] - PF::hi(w[r]));
    }

    // ---- values of masked tokens (zeros already where the loads were cut off)
    if (!whole) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (now.blk[s] >= 0 && !see.sees(now.blk[s] * kTokBlock + 4 * h + e)) {
#pragma unroll
            for (int j = 0; j < S::kVCols; ++j)
#pragma unroll
              for (int i = 0; i < S::kVWords; ++i) vr[s][e][j][i] = 0u;
          }
    }
    // ---- outputs
#pragma unroll
    for (int j = 0; j < S::kVCols; ++j) {
      if constexpr (FP8) {
        // words of four dimensions: pair the tokens' codes, then widen
#pragma unroll
        for (int i = 0; i < S::kVWords; ++i) {
          u32x4 v[4];
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2) {
            const uint32_t x = vr[e2 / 2][2 * (e2 % 2)][j][i], y = vr[e2 / 2][2 * (e2 % 2) + 1][j][i];
            const uint32_t lo = pick(x, y, 0x05010400u), hi = pick(x, y, 0x07030602u);
            v[0][e2] = PF::template from_fp8<false>(lo);
            v[1][e2] = PF::template from_fp8<true>(lo);
            v[2][e2] = PF::template from_fp8<false>(hi);
            v[3][e2] = PF::template from_fp8<true>(hi);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            acc[j][4 * i + u] = PF::mfma16(v[u], wl, PF::mfma16(v[u], w, acc[j][4 * i + u]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < S::kVWords; ++i) {
          u32x4 v[2];
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2) {
            const uint32_t x = vr[e2 / 2][2 * (e2 % 2)][j][i], y = vr[e2 / 2][2 * (e2 % 2) + 1][j][i];
            v[0][e2] = pick(x, y, kLows);
            v[1][e2] = pick(x, y, kHighs);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
            acc[j][2 * i + u] = PF::mfma16(v[u], wl, PF::mfma16(v[u], w, acc[j][2 * i + u]));
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_v(next);
    __builtin_amdgcn_sched_barrier(0);
    now = next;
    next = locate(pair + 2 * kTurn);
  }

  sum += __shfl_xor(sum, 16, 64);
  sum += __shfl_xor(sum, 32, 64);
  const int64_t part_id = (int64_t)tile * p.splits + split;
  if constexpr (OWN) {
    if (c >= rows) return;
    float* dst = p.partial + (part_id * p.part_rows + c) * p.head_dim;
#pragma unroll
    for (int j = 0; j < S::kVCols; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < S::kVDims; i += 4) {
          const int d = j * 16 * S::kVDims + (4 * h + r) * S::kVDims + i;
          if (EXACT || d < p.head_dim)
            *reinterpret_cast<f32x4*>(dst + d) = f32x4{acc[j][i][r], acc[j][i + 1][r], acc[j][i + 2][r], acc[j][i + 3][r]};
        }
    if (h == 0) *reinterpret_cast<f32x2*>(p.stats + (part_id * p.part_rows + c) * 2) = f32x2{mref, sum};
    return;
  } else {
    // ---- join the waves
    auto& part = lds->part;
    auto &part_max = lds->part_max, &part_sum = lds->part_sum;
    if (lane < kDecodeRows) {
      part_max[wave][lane] = mref;
      part_sum[wave][lane] = sum;
    }
    if (c < rows) {
#pragma unroll
      for (int j = 0; j < S::kVCols; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < S::kVDims; i += 4)
            *reinterpret_cast<f32x4*>(&part[wave][c][j * 16 * S::kVDims + (4 * h + r) * S::kVDims + i]) =
                f32x4{acc[j][i][r], acc[j][i + 1][r], acc[j][i + 2][r], acc[j][i + 3][r]};
    }
    __syncthreads();

    const int quads = p.head_dim / 4;   // fp32 quadruples of a row
    float* stats = p.stats + part_id * p.part_rows * 2;
    const rsrc_t out_r = make_rsrc(p.partial + part_id * p.part_rows * p.head_dim, (uint32_t)(p.part_rows * p.head_dim * 4));
    for (int x = threadIdx.x; x < rows * quads; x += 256) {
      const int row = EXACT ? x / (DP / 4) : x / quads, d = 4 * (x - row * quads);
      float m = part_max[0][row];
#pragma unroll
      for (int w = 1; w < kDecodeWaves; ++w) m = fmaxf(m, part_max[w][row]);
      const float base = m == kNegInf ? 0.f : m;
      float total = 0.f;
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kDecodeWaves; ++w) {
        const float f = exp2_of(part_max[w][row] - base);
        total += f * part_sum[w][row];
        const f32x4 y = *reinterpret_cast<const f32x4*>(&part[w][row][d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += f * y[i];
      }
      if (parts == 1) {
        T* dst = static_cast<T*>(p.out) + seq * p.o_ts + (head0 + row) * p.o_hs + d;
        *reinterpret_cast<u32x2*>(dst) = finish<F>(o, total, p.v_scale);
      } else {
        store16_coherent(o, out_r, (uint32_t)(row * p.head_dim + d) * 4);
        if (d == 0) {
          store_shared(stats + 2 * row, m);
          store_shared(stats + 2 * row + 1, total);
        }
      }
    }
    if (parts == 1) return;
    if (!workgroup_arrive_last(p.counters + tile, (uint32_t)parts, &lds->flag)) return;

    // ---- join the parts, in part order
    join_parts<F>(p, tile, parts, rows, [&](int r) { return seq * p.o_ts + (head0 + r) * p.o_hs; });
  }
}

// Workgroups of a compute unit by the registers that a head's accumulators and loads
// in flight take, without spills.
template <class F, class PF, bool FP8, int DP, bool EXACT>
__global__ void __launch_bounds__(256, DP == 64 ? 4 : DP == 128 ? 3 : 1) attn_decode(AttnArgs p) {
  __shared__ DecodeLds<DP> lds;
  decode_body<F, PF, FP8, DP, EXACT, false>(p, blockIdx.x + p.first_block, &lds);
}

}  // namespace
}  // namespace qg
