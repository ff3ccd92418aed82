// Causal attention of several new tokens per sequence over the paged cache.
//
// A workgroup of four waves takes 128 rows of one sequence and key-value head. A
// row is one query head of one new token, the heads of a token side by side, so
// heads that share keys share the workgroup's tiles of K and V. Each wave owns 32
// rows as the columns of 32x32x16 matrix products: scores S^T = K q^T of 64
// tokens at a time, a running maximum and sum per row in registers (fp32), and
// outputs O^T = V^T P^T.
//
// Tiles of K and V (64 tokens, four 16-token blocks of any four pages) go through
// registers into two LDS buffers in turn, one barrier per tile: wave w loads block
// w of the next tile while the current one is used.
//   K    rows of 16-byte chunks, chunk number xor token, so that the 16 tokens that
//        are read together (one chunk each) lie in different banks.
//   V    rows as in memory; the operand wants 4 consecutive tokens of one dimension
//        per lane, which the transposing LDS read gives: 16 lanes read 4 tokens of
//        16 dimensions. Its 64-byte units are permuted by token so that those 4
//        tokens lie in different banks.
//   P    the scores leave the matrix unit with row c and tokens 8x + 4h .. + 3 in
//        lane (c, h) = (lane % 32, lane / 32): two such runs are the second operand
//        of the next product as they stand, if V's tokens come in the same order.
// The weights P are rounded once to 16 bits for the matrix unit; statistics,
// sums and accumulators stay fp32.
#include "attn_device.h"

namespace qg {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_t;

constexpr int kTile = 64;                       // tokens of a tile
constexpr int kTileBlocks = kTile / kTokBlock;  // one per wave

template <int DP>
struct PrefillLds {
  static constexpr int kRow = DP * 2;             // bytes of a token
  static constexpr int kBytes = kTile * kRow;     // K or V of a tile
  static constexpr int kTotal = 4 * kBytes;       // two buffers
  // byte place of 16-byte chunk c of token t
  static __device__ __forceinline__ int k_at(int t, int c) {
    const int x = DP == 64 ? (t >> 1) & 7 : t & 15;
    return t * kRow + ((c ^ x) << 4);
  }
  static __device__ __forceinline__ int v_at(int t, int c) {
    const int x = DP == 64 ? (t >> 1) & 1 : t & 3;
    return t * kRow + ((c ^ (x << 2)) << 4);
  }
};

template <class F, class PF, bool FP8, int DP, bool EXACT>
__device__ __forceinline__ void prefill_body(const AttnArgs& p, char* lds, int* flag) {
  using L = PrefillLds<DP>;
  using T = typename F::T;
  constexpr int kElt = FP8 ? 1 : 2;
  constexpr int kLanes = DP * kElt / 16;          // lanes that load one token
  constexpr int kRows = 64 / kLanes;              // tokens of a load
  constexpr int kLoads = kTokBlock / kRows;       // loads of a block
  constexpr int kSteps = DP / 16;
  constexpr int kDB = DP / 32;

  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // key-value heads innermost: the workgroups of one head, which read the same
  // tiles, land on one XCD where there are 8 of them (or a multiple); the last
  // rows, which see most, first; parts of one row tile apart
  const int tiles = p.num_seqs * p.kv_heads * p.row_tiles;
  const int split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
  const int kv_head = tile % p.kv_heads;
  const int seq = tile / p.kv_heads % p.num_seqs;
  const int row0 = (p.row_tiles - 1 - tile / p.kv_heads / p.num_seqs) * kPrefillRows;

  const int len = min(max(scalar_load(p.lens + seq), 0), p.max_len);
  const int q0 = min(max(scalar_load(p.q_start + seq), 0), p.num_tokens);
  const int q1 = min(max(scalar_load(p.q_start + seq + 1), q0), p.num_tokens);
  const int new_tokens = min(q1 - q0, p.max_q);
  const int all_rows = new_tokens * p.group;
  if (row0 >= all_rows) return;
  const int rows = min(kPrefillRows, all_rows - row0);
  const int pos0 = len - new_tokens;              // position of the first new token
  const int pos_min = pos0 + row0 / p.group, pos_max = pos0 + (row0 + rows - 1) / p.group;
  const Visible see(max(0, pos_max + 1), p.window ? pos_min - p.window + 1 : 0, p.window ? p.sinks : 0);
  const int parts = max(1, (see.blocks + p.split_blocks - 1) / p.split_blocks);
  if (split >= parts) return;
  const int v_begin = split * p.split_blocks, v_end = min(see.blocks, v_begin + p.split_blocks);

  // ---- this lane's row, and the wave's span of positions
  const int row = row0 + wave * 32 + c;
  const bool live = row < all_rows;
  const int qi = live ? row / p.group : 0;
  const int head = kv_head * p.group + (live ? row - qi * p.group : 0);
  const int pos = live ? pos0 + qi : -1;
  const int low = p.window ? pos - p.window + 1 : 0;
  const int wave_rows = min(32, rows - wave * 32);   // may be <= 0
  const int wave_min = pos0 + (row0 + wave * 32) / p.group;
  const int wave_max = wave_rows > 0 ? pos0 + (row0 + wave * 32 + wave_rows - 1) / p.group : -1;
  const int wave_low = p.window ? wave_max - p.window + 1 : 0;   // every row of the wave sees low..min

  u32x4 q[kSteps];
  {
    const T* src = static_cast<const T*>(p.q) + (int64_t)(q0 + qi) * p.q_ts + head * p.q_hs;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = 16 * s + 8 * h;
      q[s] = u32x4{0, 0, 0, 0};
      if (live && d < p.head_dim) q[s] = *reinterpret_cast<const u32x4*>(src + d);
    }
  }

  // ---- loads: this wave's block of a tile
  const int32_t* table = p.cache.table + seq * p.cache.table_stride;
  const uint32_t ts_bytes = (uint32_t)p.cache.token_stride * kElt;
  const char* kbase = static_cast<const char*>(p.cache.k) + kv_head * p.cache.head_stride * kElt;
  const char* vbase = static_cast<const char*>(p.cache.v) + kv_head * p.cache.head_stride * kElt;
  const int l_row = lane / kLanes, l_chunk = lane % kLanes;
  const uint32_t voff = EXACT || l_chunk * 16 < p.head_dim * kElt ? l_row * ts_bytes + l_chunk * 16 : 0x80000000u;
  u32x4 kr[kLoads], vr[kLoads];
  int ld_blk = 0;
  // page of virtual block v, or -1
  auto page_at = [&](int v, int* blk, int* place) {
    const bool there = v < v_end;
    *blk = there ? see.block(v) : 0;
    const int col = page_of(p.cache, *blk, place);
    const int page = there ? scalar_load(table + col) : -1;
    return page < p.cache.num_pages ? page : -1;
  };
  auto load = [&](int v0) {
    int place;
    const int page = page_at(v0 + wave, &ld_blk, &place);
    const bool ok = page >= 0;
    const int64_t at = ok ? page * p.cache.page_stride + (int64_t)place * kTokBlock * p.cache.token_stride : 0;
    const uint32_t bytes = ok ? min(kTokBlock, see.len - ld_blk * kTokBlock) * ts_bytes : 0u;
    const rsrc_t rk = make_rsrc(kbase + at * kElt, bytes), rv = make_rsrc(vbase + at * kElt, bytes);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) kr[i] = load16(rk, voff, i * kRows * ts_bytes);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) vr[i] = load16(rv, voff, i * kRows * ts_bytes);
  };
  auto store = [&](char* buf) {
    // values that no row of the tile sees, in a block that is partly seen
    const int j0 = ld_blk * kTokBlock;
    const bool cut = !(j0 >= see.low || j0 + kTokBlock <= see.sinks);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int t = wave * kTokBlock + i * kRows + l_row;
      if (cut && !see.sees(j0 + i * kRows + l_row)) vr[i] = u32x4{0, 0, 0, 0};
      if constexpr (FP8) {
        u32x4 k[2], v[2];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          k[w / 2][2 * (w % 2)] = F::template from_fp8<false>(kr[i][w]);
          k[w / 2][2 * (w % 2) + 1] = F::template from_fp8<true>(kr[i][w]);
          v[w / 2][2 * (w % 2)] = PF::template from_fp8<false>(vr[i][w]);
          v[w / 2][2 * (w % 2) + 1] = PF::template from_fp8<true>(vr[i][w]);
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          *reinterpret_cast<u32x4*>(buf + L::k_at(t, 2 * l_chunk + w)) = k[w];
          *reinterpret_cast<u32x4*>(buf + L::kBytes + L::v_at(t, 2 * l_chunk + w)) = v[w];
        }
      } else {
        *reinterpret_cast<u32x4*>(buf + L::k_at(t, l_chunk)) = kr[i];
        *reinterpret_cast<u32x4*>(buf + L::kBytes + L::v_at(t, l_chunk)) = vr[i];
      }
    }
  };

  float mref = kNegInf, sum = 0.f;
  f32x16 acc[kDB];
#pragma unroll
  for (int d = 0; d < kDB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;

  // transposing read: lane reads 8 bytes of token (lane % 16) / 4 of its run of
  // four, dimensions 16 * (lane / 16 % 2) + 4 * (lane % 4)
  const int tr_row = 4 * h + ((lane & 15) >> 2);
  const int tr_chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), tr_low = (lane & 1) * 8;

  load(v_begin);
  if (v_begin < v_end) store(lds);
  for (int v0 = v_begin, turn = 0; v0 < v_end; v0 += kTileBlocks, turn ^= 1) {
    const char* kt = lds + turn * 2 * L::kBytes;
    const char* vt = kt + L::kBytes;
    int blk[kTileBlocks];
    bool whole = true;
#pragma unroll
    for (int b = 0; b < kTileBlocks; ++b) {
      int place;
      const int page = page_at(v0 + b, &blk[b], &place);
      if (page < 0) blk[b] = -1;
      const int j0 = blk[b] * kTokBlock;
      whole = whole && blk[b] >= 0 && j0 + kTokBlock <= wave_min + 1 && (j0 >= wave_low || j0 + kTokBlock <= p.sinks);
    }
    __syncthreads();
    load(v0 + kTileBlocks);

    // the wave's rows may all lie before the tile's tokens
    const bool any = see.block(v0) * kTokBlock <= wave_max;
    if (any) {
      f32x16 s[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          s[b] = F::mfma32(*reinterpret_cast<const u32x4*>(kt + L::k_at(32 * b + c, 2 * k + h)), q[k], s[b]);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] *= p.scale_log2;
      if (!whole) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = blk[2 * b + i / 8];   // registers 0-7: tokens of the first block
            const int j = at * kTokBlock + 8 * (i / 4 % 2) + 4 * h + i % 4;
            if (at < 0 || j > pos || (j < low && j >= p.sinks)) s[b][i] = kNegInf;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
      if (__any(top > mref + kSlack)) {
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
      const float base = mref == kNegInf ? 0.f : mref;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[b][i] = exp2_of(s[b][i] - base);
          sum += s[b][i];
        }
#pragma unroll
      for (int u = 0; u < 4; ++u) {   // 16 tokens per product
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = PF::pack(s[u / 2][8 * (u % 2) + 2 * i], s[u / 2][8 * (u % 2) + 2 * i + 1]);
#pragma unroll
        for (int d = 0; d < kDB; ++d) {
          u32x4 v;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = 16 * u + 8 * x + tr_row;
            const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4_t)(vt + L::v_at(t, 4 * d + tr_chunk) + tr_low));
            const u32x2 y = __builtin_bit_cast(u32x2, r);
            v[2 * x] = y[0];
            v[2 * x + 1] = y[1];
          }
          acc[d] = PF::mfma32(v, w, acc[d]);
        }
      }
    }
    if (v0 + kTileBlocks < v_end) store(lds + (turn ^ 1) * 2 * L::kBytes);
  }

  // ---- outputs of the wave's rows, or their part
  sum += __shfl_xor(sum, 32, 64);
  const int64_t part_id = (int64_t)tile * p.splits + split;
  if (parts == 1) {
    if (live) {
      T* dst = static_cast<T*>(p.out) + (int64_t)(q0 + qi) * p.o_ts + head * p.o_hs;
#pragma unroll
      for (int d = 0; d < kDB; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const int at = 32 * d + 2 * i + 4 * h;
          if (EXACT || at < p.head_dim)
            *reinterpret_cast<u32x2*>(dst + at) =
                finish<F>(f32x4{acc[d][i], acc[d][i + 1], acc[d][i + 2], acc[d][i + 3]}, sum, p.v_scale);
        }
    }
    return;
  }
  if (live) {
    const int r = row - row0;
    const rsrc_t out_r =
        make_rsrc(p.partial + part_id * p.part_rows * p.head_dim, (uint32_t)(p.part_rows * p.head_dim * 4));
#pragma unroll
    for (int d = 0; d < kDB; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int at = 32 * d + 2 * i + 4 * h;
        if (EXACT || at < p.head_dim)
          store16_coherent(f32x4{acc[d][i], acc[d][i + 1], acc[d][i + 2], acc[d][i + 3]}, out_r,
                           (uint32_t)(r * p.head_dim + at) * 4);
      }
    if (h == 0) {
      store_shared(p.stats + (part_id * p.part_rows + r) * 2, mref);
      store_shared(p.stats + (part_id * p.part_rows + r) * 2 + 1, sum);
    }
  }
  if (!workgroup_arrive_last(p.counters + tile, (uint32_t)parts, flag)) return;
  join_parts<F>(p, tile, parts, rows, [&](int r) {
    const int i = (row0 + r) / p.group;
    return (int64_t)(q0 + i) * p.o_ts + (int64_t)(kv_head * p.group + row0 + r - i * p.group) * p.o_hs;
  });
}

// Two workgroups of a CU where the heads fit 128 values (two waves per SIMD); the
// accumulators of longer heads take all registers of one wave per SIMD.
template <class F, class PF, bool FP8, int DP, bool EXACT>
__global__ void __launch_bounds__(256, DP <= 128 ? 2 : 1) attn_prefill(AttnArgs p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ int flag;
  prefill_body<F, PF, FP8, DP, EXACT>(p, lds, &flag);
}

template <class F, class PF, bool FP8, int DP>
hipError_t launch_exact(const AttnArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 grid((unsigned)(tiles * a.splits));
  constexpr int lds = PrefillLds<DP>::kTotal;
  if (a.head_dim == DP) hipLaunchKernelGGL((attn_prefill<F, PF, FP8, DP, true>), grid, dim3(256), lds, s, a);
  else hipLaunchKernelGGL((attn_prefill<F, PF, FP8, DP, false>), grid, dim3(256), lds, s, a);
  return hipGetLastError();
}

template <class F, class PF, bool FP8>
hipError_t launch_dim(const AttnArgs& a, int64_t tiles, hipStream_t s) {
  if (a.head_dim <= 64) return launch_exact<F, PF, FP8, 64>(a, tiles, s);
  if (a.head_dim <= 128) return launch_exact<F, PF, FP8, 128>(a, tiles, s);
  return launch_exact<F, PF, FP8, 256>(a, tiles, s);
}

}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& a, bool bf16, bool fp8, int64_t tiles, hipStream_t s) {
  if (bf16) return fp8 ? launch_dim<BF16, F16, true>(a, tiles, s) : launch_dim<BF16, BF16, false>(a, tiles, s);
  return fp8 ? launch_dim<F16, F16, true>(a, tiles, s) : launch_dim<F16, F16, false>(a, tiles, s);
}

}  // namespace qg
