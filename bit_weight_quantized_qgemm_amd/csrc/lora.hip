// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + s[a] * B[a] (A[a] x[t]),  a = ids[t].
//
// Rows are sorted by adapter once per batch (lora_plan), so that a tile holds rows of
// one adapter; then two launches per projection: A x (lora_shrink), and its product with
// B, added to the base (lora_expand). A batch of single tokens is bound by the adapters'
// bytes, prompts by x, base and out. Measured on MI355X, us, both launches of a captured call
// (floor: bytes at 5.13 TB/s, the rate of a large copy):
//   1 row, 4096 to 4096, rank 16, fp16                                  9.1  (0.06)
//   64 rows of 64 adapters, 8192 to 8192 + 1024 + 1024, rank 16, bf16  21.2  (14.6)
//   128 rows of 24 adapters of ranks 8..64, 8192 to 28672, fp16        27.9  (13.2)
//   1003 rows of 5 adapters, 4096 to 11008, rank 64, fp16              29.4  (12.1)
//   8192 rows of 3 adapters, 8192 to 8192, rank 16, bf16               95.6  (78.8)
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
// are its own whatever tile it is in. One workgroup: the work is a few loads per row, and
// it is done once for all projections of all layers (3 to 5 us up to 1003 rows, 10 for 8192, 59
// for 65535 of 4096 adapters).
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
__device__ __forceinline__ LoraTile lora_tile(const LoraArgs& p, int tile, int tiles_at, int count_at) {
  const int32_t* at = p.plan + tiles_at + 4 * tile;
  LoraTile t{scalar_load(at), scalar_load(at + 1), scalar_load(at + 2), p.rank};
  // a plan of other numbers of rows and adapters is not followed
  const bool fits = scalar_load(p.plan) == p.tokens && scalar_load(p.plan + 1) == p.adapters;
  if (!fits || tile >= scalar_load(p.plan + count_at)) t.rows = 0;
  if (t.rows > 0 && t.adapter >= 0 && p.ranks)
    t.rank = (min(max(scalar_load(p.ranks + t.adapter), 0), p.rank) + 7) / 8 * 8;
  return t;
}

// y = A x: RB * 16 rows by NT * 16 ranks of one adapter, over a part of K. The four waves
// take a quarter of the part each and meet in LDS; the last workgroup of a tile to arrive
// adds the parts, in order. Ranks are the rows of the product (first operand) and tokens
// its columns, so that a lane ends with four ranks of one token; both operands go from
// memory to registers as they stand. Rows and ranks that do not exist repeat the last
// one's loads and are dropped at the end.
//
// Bound by memory, behind a chain of launch, plan entry, rows and first loads and before the
// parts' join: 64 rows of 64 adapters at 48 ranks of 8192 take 12.3 us for 51 MB (4.1 TB/s),
// 8192 rows of 8192 at rank 16 39 us for 134 MB, which a bare read takes in 22: without the
// loads of x the latter took 10.6 us of then 39.8.
template <class F, int RB, int NT>
__global__ void __launch_bounds__(256) lora_shrink(LoraArgs p) {
  constexpr int kUnroll = RB == 1 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) float part[kLoraWaves][RB * NT][64][4];
  __shared__ int flag;
  const int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // parts of a tile stand side by side; workgroups of the same rows and values (chunks of
  // ranks) are eight apart, on one XCD, whose cache they share
  const uint32_t run = blockIdx.x / (8u * p.chunks), in_run = blockIdx.x - run * (8u * p.chunks);
  const int chunk = in_run / 8, part_no = run * 8 + in_run % 8;
  const int tile_no = part_no / p.splits, split = part_no - tile_no * p.splits;
  if (tile_no >= (RB == 1 ? p.cap16 : p.cap64)) return;
  const LoraTile t = RB == 1 ? lora_tile(p, tile_no, p.tiles16, 2) : lora_tile(p, tile_no, p.tiles64, 3);
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
  const int begin = split * p.split_k, end = min(begin + p.split_k, p.k);
  // Runs of kUnroll steps go to the waves in turn, so that a workgroup reads rows in long
  // stretches; one run's loads stand in flight beside the products of the one before.
  struct Steps {
    u32x4 x[kUnroll][RB], a[kUnroll][NT];
  };
  auto load = [&](Steps& o, int run) {
    const int k = begin + run * (32 * kUnroll) + 8 * h;
#pragma unroll
    for (int s = 0; s < kUnroll; ++s) {
#pragma unroll
      for (int i = 0; i < NT; ++i) o.a[s][i] = *reinterpret_cast<const u32x4*>(ap[i] + k + 32 * s);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        // up to two tiles of ranks are all there are: x is read once, and left out of the
        // caches where it is long (8192 rows, rank 16: 96.7 us, 98.8 without the hint)
        const u32x4* at = reinterpret_cast<const u32x4*>(xp[b] + k + 32 * s);
        o.x[s][b] = RB == 4 && NT <= 2 ? __builtin_nontemporal_load(at) : *at;
      }
    }
  };
  auto multiply = [&](const Steps& o) {
#pragma unroll
    for (int s = 0; s < kUnroll; ++s)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b][i] = F::mfma16(o.a[s][i], o.x[s][b], acc[b][i]);
  };
  const int runs = (end - begin) / (32 * kUnroll);
  Steps even, odd;
  if (wave < runs) load(even, wave);
  for (int r = wave; r < runs; r += 2 * kLoraWaves) {
    if (r + kLoraWaves < runs) load(odd, r + kLoraWaves);
    multiply(even);
    if (r + 2 * kLoraWaves < runs) load(even, r + 2 * kLoraWaves);
    if (r + kLoraWaves < runs) multiply(odd);
  }
  // what is left, step by step; the end of K may be within one
  for (int k0 = begin + (runs * kUnroll + wave) * 32; k0 < end; k0 += kLoraWaves * 32) {
    const int k = k0 + 8 * h;
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
  constexpr uint32_t kPartBytes = RB * NT * 64 * 16;
  const int64_t first_part = ((int64_t)tile_no * p.chunks + chunk) * p.splits;
  const rsrc_t mine = make_rsrc(p.partial + (first_part + split) * (kPartBytes / 4), kPartBytes);
  auto finish_tile = [&](int x, f32x4 y) {
    const int at = chunk * NT + x % NT, row = x / NT * 16 + c, r0 = at % p.rank_tiles * 16 + 4 * h;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i >= t.rank) y[i] = 0.f;
    if (at < tiles && row < t.rows)
      *reinterpret_cast<f32x4*>(p.y + ((int64_t)(t.first + row) * tiles + at) * 16 + 4 * h) = y;
  };
#pragma unroll
  for (int n = 0; n < (RB * NT + 3) / 4; ++n) {
    const int x = n * kLoraWaves + wave;
    if (x < RB * NT) {
      f32x4 y = *reinterpret_cast<const f32x4*>(part[0][x][lane]);
#pragma unroll
      for (int w = 1; w < kLoraWaves; ++w) {
        const f32x4 z = *reinterpret_cast<const f32x4*>(part[w][x][lane]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] += z[i];
      }
      if (p.splits == 1) finish_tile(x, y);
      else store16_coherent(y, mine, (uint32_t)(x * 64 + lane) * 16);
    }
  }
  if (p.splits == 1) return;
  if (!workgroup_arrive_last(p.counters + tile_no * p.chunks + chunk, (uint32_t)p.splits, &flag)) return;
#pragma unroll
  for (int n = 0; n < (RB * NT + 3) / 4; ++n) {
    const int x = n * kLoraWaves + wave;
    if (x < RB * NT) {
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
      for (int s0 = 0; s0 < p.splits; s0 += 8) {   // eight parts in flight
        f32x4 z[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          z[u] = load16_coherent(make_rsrc(p.partial + (first_part + min(s0 + u, p.splits - 1)) * (kPartBytes / 4), kPartBytes),
                                 (uint32_t)(x * 64 + lane) * 16);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] += s0 + u < p.splits ? z[u][i] : 0.f;
      }
      finish_tile(x, y);
    }
  }
}

// out = base + s * B y: a wave takes a tile of RB * 16 rows and 64 columns at a time, the
// four waves of a workgroup columns next to each other. Columns are the rows of the
// product and tokens its columns: row i of block j stands for column 32 (j / 2) + 8 (i / 4)
// + 4 (j % 2) + i % 4, so that a lane ends with eight consecutive columns of one token
// twice, and four lanes with 64 bytes. y is brought into range by a power of two per token
// (fp16: near 1) and goes in as two 16-bit terms (the rounded value and the rest, good to
// 2^-22 or 2^-16 of it), each with a product of its own. Ranks up to 16 leave half of a
// product's inner length of 32 free: there the terms lie one after the other, against B
// twice (PAIRED), and cost one product. KS: steps of 32 ranks.
//
// Bound by base, out and B: 8192 rows of 8192 columns at rank 16 take 55 us for 268 MB (4.9
// TB/s, a copy's rate). Rows of B lie 2 * rank bytes apart, so where an adapter of rank 8 or
// 16 lies in a pool of rank 64 its whole lines of 128 bytes are moved: 128 rows of 21 such
// adapters on 28672 columns take 18 us for 14 MB of base and out and 77 MB of lines (counted
// at the L2), of which the product uses 40.
//
// An infinite value of B times a rest of 0, or of the other sign than its first term, would
// make NaN of a sum that is infinite, and so would a rest's product that passes the end beside
// a first term's. So a value that is not 0 has a first term that is not (the smallest normal
// one, less which the rest then is), and a sum that comes out NaN is taken from the first terms
// alone, which are infinite, or NaN, where the formula is (behind the stores: 64 rows of 64
// adapters 20.0 us a call, 19.8 without the look, other cases the same; between products and
// stores 128 rows on 28672 columns took 28.5 instead of 27.5). The launch bounds keep the waves
// that this would cost (128 rows 30.2 with four per SIMD instead of five, 64 rows 20.5 with
// six instead of eight).
template <class F, int RB, int KS, bool PAIRED>
__global__ void __launch_bounds__(256, KS > 2 ? 1 : RB == 1 ? (KS == 1 ? 8 : 5) : (KS == 1 ? 4 : 3)) lora_expand(LoraArgs p) {
  constexpr bool kHalf = std::is_same_v<F, F16>;
  constexpr uint32_t kSmallest = kHalf ? 0x0400u : 0x0080u;   // normal value
  const int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroups that run together take the columns of the same rows (8192 rows, 8192 to 8192,
  // rank 16, four tiles of columns to a wave: 61 us, 69 where they take the rows of the same
  // columns)
  const uint32_t groups = p.group_begin[p.slices];
  const int tile_no = blockIdx.x / groups, group = blockIdx.x - tile_no * groups;
  const LoraTile t = RB == 1 ? lora_tile(p, tile_no, p.tiles16, 2) : lora_tile(p, tile_no, p.tiles64, 3);
  if (t.rows <= 0 || (t.adapter < 0 && p.in_place)) return;
  using T = typename F::T;

  int slice = 0;
  while (slice + 1 < p.slices && group >= p.group_begin[slice + 1]) ++slice;
  const int col_end = p.col_begin[slice + 1];
  const int first_col = p.col_begin[slice] + (group - p.group_begin[slice]) * p.group_cols * kLoraCols;
  const int group_end = min(col_end, first_col + p.group_cols * kLoraCols);
  int col = first_col + wave * kLoraCols;
  const bool mine = col < group_end;   // this wave has columns

  const T* base_row[RB];
  T* out_row[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int64_t row = p.plan[16 + t.first + min(16 * b + c, t.rows - 1)];
    base_row[b] = static_cast<const T*>(p.base) + row * p.base_stride + 8 * h;
    out_row[b] = static_cast<T*>(p.out) + row * p.out_stride + 8 * h;
  }
  u32x4 base[RB][2];
  auto load_base = [&](int at) {
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        base[b][x] = u32x4{0, 0, 0, 0};
        if (p.base && 16 * b < t.rows && at + 32 * x + 8 * h < col_end)
          base[b][x] = *reinterpret_cast<const u32x4*>(base_row[b] + at + 32 * x);
      }
  };
  if (mine) load_base(col);

  // ---- B: the eight of ranks of this lane in each step
  const int eights = t.adapter < 0 ? 0 : t.rank / 8;
  const T* b_rows = static_cast<const T*>(p.b) + max(0, t.adapter) * p.b_stride;
  int chunk[KS];   // -1: none
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int q = 4 * s + h;
    chunk[s] = q < eights ? q : PAIRED && q < 2 * eights ? q - eights : -1;
  }
  u32x4 w[4][KS];
  auto load_b = [&](int at) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = at + 32 * (j / 2) + 8 * (c / 4) + 4 * (j % 2) + c % 4;
      const T* b_row = b_rows + (int64_t)min(n, col_end - 1) * p.rank;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        w[j][s] = u32x4{0, 0, 0, 0};
        if (chunk[s] >= 0) w[j][s] = *reinterpret_cast<const u32x4*>(b_row + chunk[s] * 8);
      }
    }
  };
  if (mine) load_b(col);

  // ---- y as the second operand, in LDS: both terms of each step, or (PAIRED) the two in one.
  // Wave w prepares row blocks w, w + 4, ...
  __shared__ __attribute__((aligned(16))) u32x4 terms[RB][KS][PAIRED ? 1 : 2][64];
  __shared__ float factors[RB][16];
#pragma unroll
  for (int n = 0; n < (RB + kLoraWaves - 1) / kLoraWaves; ++n) {
    const int b = n * kLoraWaves + wave;
    if (b >= RB || 16 * b >= t.rows || t.adapter < 0) continue;
    f32x4 v[KS][2];
    const float* src = p.y + ((int64_t)(t.first + min(16 * b + c, t.rows - 1)) * p.slices + slice) * p.rank_tiles * 16;
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        v[s][x] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (chunk[s] >= 0) v[s][x] = *reinterpret_cast<const f32x4*>(src + chunk[s] * 8 + 4 * x);
      }
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(v[s][x][e]));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    // 2^exponent <= top < 2^(exponent + 1) for normal values; an infinite or NaN sum stays what
    // it is, the rest of an infinite one is 0. fp16 is brought near 1, as far as the factors are
    // normal. bf16 has fp32's range, in which B times 1 may pass the end where B y does not: it
    // stays as it is between 2^-60, whose rests are normal, and 2^120, whose first terms are finite
    const int exponent = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
    const int e = kHalf ? min(max(exponent, -100), 100) : exponent - min(max(exponent, -60), 119);
    const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
    if (h == 0) factors[b][c] = (p.scales ? p.scales[t.adapter] : 1.f) * __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4 hi, lo;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float v0 = v[s][x][2 * i] * down, v1 = v[s][x][2 * i + 1] * down;
          hi[2 * x + i] = F::pack(v0, v1);
          if (v[s][x][2 * i] != 0.f && !(hi[2 * x + i] & 0x7FFFu)) hi[2 * x + i] |= kSmallest;
          if (v[s][x][2 * i + 1] != 0.f && !(hi[2 * x + i] & 0x7FFF0000u)) hi[2 * x + i] |= kSmallest << 16;
          const float h0 = F::lo(hi[2 * x + i]), h1 = F::hi(hi[2 * x + i]);
          lo[2 * x + i] = F::pack(isinf(h0) ? 0.f : v0 - h0, isinf(h1) ? 0.f : v1 - h1);
        }
      if constexpr (PAIRED) {
        terms[b][s][0][lane] = h >= eights ? lo : hi;
      } else {
        terms[b][s][0][lane] = hi;
        terms[b][s][1][lane] = lo;
      }
    }
  }
  __syncthreads();
  if (!mine) return;

  // ---- columns; true where a sum is NaN. again: such sums from the first terms alone
  auto columns = [&](auto again) {
    bool nan = false;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (16 * b < t.rows) {
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
          if (4 * s < eights) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[j] = F::mfma16(w[j][s], terms[b][s][0][lane], acc[j]);
              if constexpr (!PAIRED) acc[j] = F::mfma16(w[j][s], terms[b][s][1][lane], acc[j]);
            }
          }
        if constexpr (decltype(again)::value) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f32x4 first = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s)   // PAIRED: lanes h >= eights hold rests
              if (4 * s < eights)
                first = F::mfma16(!PAIRED || h < eights ? w[j][s] : u32x4{0, 0, 0, 0}, terms[b][s][0][lane], first);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (acc[j][i] != acc[j][i]) acc[j][i] = first[i];
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) nan |= acc[j][i] != acc[j][i];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          u32x4 o = base[b][x];   // as it is without an adapter
          if (t.adapter >= 0) {
            const float factor = factors[b][c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const f32x4 v = acc[2 * x + i / 2];
              o[i] = F::pack(F::lo(base[b][x][i]) + factor * v[2 * (i % 2)], F::hi(base[b][x][i]) + factor * v[2 * (i % 2) + 1]);
            }
          }
          if (16 * b + c < t.rows && col + 32 * x + 8 * h < col_end)
            *reinterpret_cast<u32x4*>(out_row[b] + col + 32 * x) = o;
        }
      }
    }
    return nan;
  };
  for (;;) {
    if (__builtin_expect(__any(columns(std::false_type())), 0)) columns(std::true_type());
    col += kLoraWaves * kLoraCols;
    const bool more = col < group_end;
    if (more) {
      load_base(col);
      load_b(col);
    }
    if (!more) break;
  }
}

template <class F, int RB>
void shrink_tiles(const LoraArgs& a, int chunk_tiles, dim3 grid, hipStream_t s) {
  if (chunk_tiles == 1) hipLaunchKernelGGL((lora_shrink<F, RB, 1>), grid, dim3(256), 0, s, a);
  else if (chunk_tiles == 2) hipLaunchKernelGGL((lora_shrink<F, RB, 2>), grid, dim3(256), 0, s, a);
  else if (chunk_tiles == 3) hipLaunchKernelGGL((lora_shrink<F, RB, 3>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((lora_shrink<F, RB, 4>), grid, dim3(256), 0, s, a);
}

template <class F, int KS, bool PAIRED>
void expand_tiles(const LoraArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tall_b ? a.cap64 : a.cap16) * a.group_begin[a.slices]));
  if (a.tall_b) hipLaunchKernelGGL((lora_expand<F, 4, KS, PAIRED>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((lora_expand<F, 1, KS, PAIRED>), grid, dim3(256), 0, s, a);
}

template <class F>
void expand_ranks(const LoraArgs& a, hipStream_t s) {
  if (a.rank <= 16) expand_tiles<F, 1, true>(a, s);
  else if (a.rank <= 32) expand_tiles<F, 1, false>(a, s);
  else if (a.rank <= 64) expand_tiles<F, 2, false>(a, s);
  else if (a.rank <= 128) expand_tiles<F, 4, false>(a, s);
  else expand_tiles<F, 8, false>(a, s);
}

}  // namespace

hipError_t launch_lora_plan(const LoraPlanArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(lora_plan, dim3(1), dim3(kPlanThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_lora_shrink(const LoraArgs& a, bool bf16, int chunk_tiles, hipStream_t s) {
  const dim3 grid((unsigned)(((a.tall_a ? a.cap64 : a.cap16) * a.splits + 7) / 8 * 8 * a.chunks));
  if (a.tall_a) bf16 ? shrink_tiles<BF16, 4>(a, chunk_tiles, grid, s) : shrink_tiles<F16, 4>(a, chunk_tiles, grid, s);
  else bf16 ? shrink_tiles<BF16, 1>(a, chunk_tiles, grid, s) : shrink_tiles<F16, 1>(a, chunk_tiles, grid, s);
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraArgs& a, bool bf16, hipStream_t s) {
  bf16 ? expand_ranks<BF16>(a, s) : expand_ranks<F16>(a, s);
  return hipGetLastError();
}

}  // namespace qg
