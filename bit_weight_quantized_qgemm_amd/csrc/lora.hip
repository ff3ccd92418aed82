// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + s[a] * B[a] (A[a] x[t]),  a = ids[t].
//
// Rows are sorted by adapter once per batch (lora_plan), so that a tile holds rows of
// one adapter; then two launches per projection: A x (lora_shrink), and its product with
// B, added to the base (lora_expand). A batch of single tokens is bound by the adapters'
// bytes, prompts by x, base and out.
#include "attn_device.h"
#include "lora_internal.h"

#include <type_traits>

namespace qg {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanEach = (kMaxLoraAdapters + 1 + kPlanThreads - 1) / kPlanThreads;   // adapters per thread

// A counting sort by one workgroup: rows per adapter, their prefix sums (of rows and of
// tiles), then every row to its place. Where rows of one adapter stand among each other
// is left to the order of the LDS atomics: no output depends on it, since a row's sums
// are its own whatever tile it is in.
__global__ void __launch_bounds__(kPlanThreads) lora_plan(LoraPlanArgs p) {
  __shared__ int32_t count[kMaxLoraAdapters + 1], start[kMaxLoraAdapters + 1], first_tile[kMaxLoraAdapters + 1];
  __shared__ int32_t wave_rows[kPlanThreads / 64], wave_tiles[kPlanThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, buckets = p.adapters + 1;
  for (int a = tid; a < buckets; a += kPlanThreads) count[a] = 0;
  __syncthreads();
  auto bucket_of = [&](int t) {
    const int id = p.ids[t];
    return id >= 0 && id < p.adapters ? id : p.adapters;
  };
  for (int t = tid; t < p.tokens; t += kPlanThreads) atomicAdd(&count[bucket_of(t)], 1);
  __syncthreads();
  // tiles of 16 rows in the low half of a word (at most 8192), of 64 in the high one
  int mine[kPlanEach], rows = 0, tiles = 0;
#pragma unroll
  for (int i = 0; i < kPlanEach; ++i) {
    const int a = tid * kPlanEach + i;
    mine[i] = a < buckets ? count[a] : 0;
    rows += mine[i];
    tiles += (mine[i] + 15) / 16 + ((mine[i] + 63) / 64 << 16);
  }
  int rows_to = rows, tiles_to = tiles;   // inclusive sums
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int r = __shfl_up(rows_to, d, 64), t = __shfl_up(tiles_to, d, 64);
    if (lane >= d) {
      rows_to += r;
      tiles_to += t;
    }
  }
  if (lane == 63) {
    wave_rows[wave] = rows_to;
    wave_tiles[wave] = tiles_to;
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    rows_to += wave_rows[w];
    tiles_to += wave_tiles[w];
  }
  int row = rows_to - rows, tile = tiles_to - tiles;
#pragma unroll
  for (int i = 0; i < kPlanEach; ++i) {
    const int a = tid * kPlanEach + i;
    if (a < buckets) {
      start[a] = row;
      first_tile[a] = tile;
      count[a] = 0;   // rows placed, below
    }
    row += mine[i];
    tile += (mine[i] + 15) / 16 + ((mine[i] + 63) / 64 << 16);
  }
  if (tid == kPlanThreads - 1) {
    p.plan[0] = p.tokens;
    p.plan[1] = p.adapters;
    p.plan[2] = tile & 0xFFFF;
    p.plan[3] = tile >> 16;
  }
  __syncthreads();
  for (int t = tid; t < p.tokens; t += kPlanThreads) {
    const int b = bucket_of(t), at = atomicAdd(&count[b], 1);
    const int end = b + 1 < buckets ? start[b + 1] : p.tokens;
    const int all = end - start[b], adapter = b < p.adapters ? b : -1;
    p.plan[16 + start[b] + at] = t;
    if (at % 16 == 0)
      reinterpret_cast<i32x4*>(p.plan + p.tiles16)[(first_tile[b] & 0xFFFF) + at / 16] =
          i32x4{adapter, start[b] + at, min(16, all - at), 0};
    if (at % 64 == 0)
      reinterpret_cast<i32x4*>(p.plan + p.tiles64)[(first_tile[b] >> 16) + at / 64] =
          i32x4{adapter, start[b] + at, min(64, all - at), 0};
  }
}

// A tile of sorted rows, and its adapter's rank in whole eights; rows 0 where there is none.
struct LoraTile {
  int adapter, first, rows, rank;
};
__device__ __forceinline__ LoraTile lora_tile(const LoraArgs& p, int tile) {
  const int32_t* at = p.plan + p.tiles_at + 4 * tile;
  LoraTile t{scalar_load(at), scalar_load(at + 1), scalar_load(at + 2), p.rank};
  // a plan of other numbers of rows and adapters is not followed
  const bool fits = scalar_load(p.plan) == p.tokens && scalar_load(p.plan + 1) == p.adapters;
  if (!fits || tile >= scalar_load(p.plan + (p.wide ? 3 : 2))) t.rows = 0;
  if (t.rows > 0 && t.adapter >= 0 && p.ranks)
    t.rank = (min(max(scalar_load(p.ranks + t.adapter), 0), p.rank) + 7) / 8 * 8;
  return t;
}

// y[row][16 i ..] += A x over a part of K: RB * 16 rows by NT * 16 ranks of one adapter.
// The four waves take a quarter of the part each and meet in LDS. Ranks are the rows of
// the product (first operand) and tokens its columns, so that a lane ends with four ranks
// of one token; both operands go from memory to registers as they stand. Rows and ranks
// that do not exist repeat the last one's loads and are dropped at the end.
template <class F, int RB, int NT>
__global__ void __launch_bounds__(256) lora_shrink(LoraArgs p) {
  constexpr int kUnroll = RB == 1 ? (NT == 1 ? 8 : 4) : 2;
  __shared__ __attribute__((aligned(16))) float part[kLoraWaves][RB * NT][64][4];
  const int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile_no = blockIdx.x % (uint32_t)p.cap, rest = blockIdx.x / (uint32_t)p.cap;
  const int chunk = rest % p.chunks, split = rest / p.chunks;
  const LoraTile t = lora_tile(p, tile_no);
  if (t.rows <= 0 || t.adapter < 0) return;
  using T = typename F::T;
  const int tiles = p.slices * p.rank_tiles;

  const T* xp[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int row = p.plan[16 + t.first + min(16 * b + c, t.rows - 1)];
    xp[b] = static_cast<const T*>(p.x) + row * p.x_stride;
  }
  const T* ap[NT];
  const T* adapter = static_cast<const T*>(p.a) + t.adapter * p.a_stride;
  bool any = false;   // some tile of ranks is there
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int at = min(chunk * NT + i, tiles - 1), slice = at / p.rank_tiles, r0 = (at - slice * p.rank_tiles) * 16;
    any = any || r0 < t.rank;
    ap[i] = adapter + (int64_t)(slice * p.rank + max(0, min(r0 + c, t.rank - 1))) * p.k;
  }
  if (!any) return;   // nothing reads these ranks

  f32x4 acc[RB][NT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int begin = split * p.split_k + wave * (p.split_k / kLoraWaves);
  const int end = min(begin + p.split_k / kLoraWaves, p.k);
  int k = begin + 8 * h;
  auto steps = [&](auto count) {
    constexpr int n = decltype(count)::value;
    u32x4 xr[n][RB], ar[n][NT];
#pragma unroll
    for (int s = 0; s < n; ++s) {
#pragma unroll
      for (int i = 0; i < NT; ++i) ar[s][i] = *reinterpret_cast<const u32x4*>(ap[i] + k + 32 * s);
#pragma unroll
      for (int b = 0; b < RB; ++b) xr[s][b] = *reinterpret_cast<const u32x4*>(xp[b] + k + 32 * s);
    }
#pragma unroll
    for (int s = 0; s < n; ++s)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b][i] = F::mfma16(ar[s][i], xr[s][b], acc[b][i]);
    k += 32 * n;
  };
  int left = (end - begin) / 32;   // may be negative
  for (; left >= kUnroll; left -= kUnroll) steps(std::integral_constant<int, kUnroll>{});
  for (; left > 0; --left) steps(std::integral_constant<int, 1>{});
  if (end > begin && (end - begin) % 32 != 0) {   // the end of K, no whole step
    const bool there = k < end;
    u32x4 xr[RB], ar[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      ar[i] = u32x4{0, 0, 0, 0};
      if (there) ar[i] = *reinterpret_cast<const u32x4*>(ap[i] + k);
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      xr[b] = u32x4{0, 0, 0, 0};
      if (there) xr[b] = *reinterpret_cast<const u32x4*>(xp[b] + k);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[b][i] = F::mfma16(ar[i], xr[b], acc[b][i]);
  }

#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4*>(part[wave][b * NT + i][lane]) = acc[b][i];
  __syncthreads();
  for (int x = wave; x < RB * NT; x += kLoraWaves) {
    f32x4 y = *reinterpret_cast<const f32x4*>(part[0][x][lane]);
#pragma unroll
    for (int w = 1; w < kLoraWaves; ++w) {
      const f32x4 z = *reinterpret_cast<const f32x4*>(part[w][x][lane]);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += z[i];
    }
    const int at = chunk * NT + x % NT, row = x / NT * 16 + c, r0 = at % p.rank_tiles * 16 + 4 * h;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i >= t.rank) y[i] = 0.f;
    if (at < tiles && row < t.rows)
      *reinterpret_cast<f32x4*>(p.partial + (((int64_t)split * p.tokens + t.first + row) * tiles + at) * 16 + 4 * h) = y;
  }
}

// out = base + s * B y for RB * 16 rows of one adapter and 64 columns at a time per wave.
// Columns are the rows of the product and tokens its columns: row i of block j stands for
// column 16 (i / 4) + 4 j + i % 4, so that a lane ends with 16 consecutive columns of one
// token. y is brought near 1 by a power of two per token and goes in as two 16-bit terms
// (the rounded value and the rest, good to 2^-22 or 2^-16 of it): they lie one after the
// other along the product's inner length, against B twice, so that ranks up to 16 take no
// more products for it. KS: steps of 32 of that length.
template <class F, int RB, int KS>
__global__ void __launch_bounds__(256) lora_expand(LoraArgs p) {
  const int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int parts = p.wide ? 4 / RB : 1;   // workgroups of a tile's rows
  const int tile_no = blockIdx.x % (uint32_t)p.cap, rest = blockIdx.x / (uint32_t)p.cap;
  const int row_part = rest % parts, group = rest / parts;
  LoraTile t = lora_tile(p, tile_no);
  const int skip = row_part * RB * 16;
  t.first += skip;
  t.rows = min(t.rows - skip, RB * 16);
  if (t.rows <= 0 || (t.adapter < 0 && p.in_place)) return;
  using T = typename F::T;

  int slice = 0;
  while (slice + 1 < p.slices && group >= p.group_begin[slice + 1]) ++slice;
  const int col_end = p.col_begin[slice + 1];
  int col = p.col_begin[slice] + ((group - p.group_begin[slice]) * p.group_cols + wave) * kLoraCols;
  const int group_end = min(col_end, p.col_begin[slice] + (group - p.group_begin[slice] + 1) * p.group_cols * kLoraCols);

  int64_t row[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) row[b] = p.plan[16 + t.first + min(16 * b + c, t.rows - 1)];

  // ---- y as the second operand
  const int eights = t.adapter < 0 ? 0 : t.rank / 8;   // of ranks
  u32x4 y[RB][KS];
  float factor[RB];
  int chunk[KS];   // eight of ranks of this lane in each step; -1: none
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int q = 4 * s + h;
    chunk[s] = q < eights ? q : q < 2 * eights ? q - eights : -1;
  }
  const float scale = t.adapter < 0 || !p.scales ? 1.f : p.scales[t.adapter];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    f32x4 v[KS][2];
    const int r = t.first + min(16 * b + c, t.rows - 1);
    const int64_t row_elems = (int64_t)p.slices * p.rank_tiles * 16;
    const float* src = p.partial + r * row_elems + slice * p.rank_tiles * 16;
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      v[s][0] = v[s][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (chunk[s] >= 0) {
        for (int u = 0; u < p.splits; ++u) {
          const f32x4* z = reinterpret_cast<const f32x4*>(src + u * p.tokens * row_elems + chunk[s] * 8);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[s][x][i] += z[x][i];
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(v[s][x][i]));
    }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    // 2^e <= top < 2^(e+1) for normal values; an infinite or NaN sum stays what it is
    const int e = min(max((int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127, -100), 100);
    const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
    factor[b] = scale * __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const bool rest_of = 4 * s + h >= eights;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float v0 = v[s][x][2 * i] * down, v1 = v[s][x][2 * i + 1] * down;
          const uint32_t hi = F::pack(v0, v1);
          y[b][s][2 * x + i] = rest_of ? F::pack(v0 - F::lo(hi), v1 - F::hi(hi)) : hi;
        }
    }
  }

  // ---- columns
  const T* b0 = static_cast<const T*>(p.b) + max(0, t.adapter) * p.b_stride;
  for (; col < group_end; col += kLoraWaves * kLoraCols) {
    f32x4 acc[RB][4];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[b][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 base[RB][2];
    const int mine = col + 16 * h;   // this lane's columns
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        base[b][x] = u32x4{0, 0, 0, 0};
        if (p.base && mine + 8 * x < col_end)
          base[b][x] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.base) + row[b] * p.base_stride + mine + 8 * x);
      }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if (4 * s < 2 * eights) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = min(col + 16 * (c / 4) + 4 * j + c % 4, col_end - 1);
          u32x4 w = {0, 0, 0, 0};
          if (chunk[s] >= 0) w = *reinterpret_cast<const u32x4*>(b0 + (int64_t)n * p.rank + chunk[s] * 8);
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[b][j] = F::mfma16(w, y[b][s], acc[b][j]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        u32x4 o = base[b][x];   // as it is without an adapter
        if (t.adapter >= 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 v = acc[b][2 * x + i / 2];
            o[i] = F::pack(F::lo(base[b][x][i]) + factor[b] * v[2 * (i % 2)],
                           F::hi(base[b][x][i]) + factor[b] * v[2 * (i % 2) + 1]);
          }
        }
        if (16 * b + c < t.rows && mine + 8 * x < col_end)
          *reinterpret_cast<u32x4*>(static_cast<T*>(p.out) + row[b] * p.out_stride + mine + 8 * x) = o;
      }
  }
}

template <class F, int RB>
void shrink_tiles(const LoraArgs& a, int chunk_tiles, dim3 grid, hipStream_t s) {
  if (chunk_tiles == 1) hipLaunchKernelGGL((lora_shrink<F, RB, 1>), grid, dim3(256), 0, s, a);
  else if (chunk_tiles == 2) hipLaunchKernelGGL((lora_shrink<F, RB, 2>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((lora_shrink<F, RB, 4>), grid, dim3(256), 0, s, a);
}

// Tiles of 64 rows stay whole while y fits the registers beside the sums (ranks up to 64).
template <class F>
void expand_ranks(const LoraArgs& a, unsigned blocks, hipStream_t s) {
  const int steps = (a.rank + 15) / 16;
  if (a.wide && steps <= 1) hipLaunchKernelGGL((lora_expand<F, 4, 1>), dim3(blocks), dim3(256), 0, s, a);
  else if (a.wide && steps <= 2) hipLaunchKernelGGL((lora_expand<F, 4, 2>), dim3(blocks), dim3(256), 0, s, a);
  else if (a.wide && steps <= 4) hipLaunchKernelGGL((lora_expand<F, 4, 4>), dim3(blocks), dim3(256), 0, s, a);
  else {
    const dim3 grid(blocks * (a.wide ? 4 : 1));
    if (steps <= 1) hipLaunchKernelGGL((lora_expand<F, 1, 1>), grid, dim3(256), 0, s, a);
    else if (steps <= 2) hipLaunchKernelGGL((lora_expand<F, 1, 2>), grid, dim3(256), 0, s, a);
    else if (steps <= 4) hipLaunchKernelGGL((lora_expand<F, 1, 4>), grid, dim3(256), 0, s, a);
    else if (steps <= 8) hipLaunchKernelGGL((lora_expand<F, 1, 8>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((lora_expand<F, 1, 16>), grid, dim3(256), 0, s, a);
  }
}

}  // namespace

hipError_t launch_lora_plan(const LoraPlanArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(lora_plan, dim3(1), dim3(kPlanThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_lora_shrink(const LoraArgs& a, bool bf16, int chunk_tiles, hipStream_t s) {
  const dim3 grid((unsigned)(a.cap * a.chunks * a.splits));
  if (a.wide) bf16 ? shrink_tiles<BF16, 4>(a, chunk_tiles, grid, s) : shrink_tiles<F16, 4>(a, chunk_tiles, grid, s);
  else bf16 ? shrink_tiles<BF16, 1>(a, chunk_tiles, grid, s) : shrink_tiles<F16, 1>(a, chunk_tiles, grid, s);
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraArgs& a, bool bf16, hipStream_t s) {
  const unsigned blocks = (unsigned)(a.cap * a.group_begin[a.slices]);
  bf16 ? expand_ranks<BF16>(a, blocks, s) : expand_ranks<F16>(a, blocks, s);
  return hipGetLastError();
}

}  // namespace qg
