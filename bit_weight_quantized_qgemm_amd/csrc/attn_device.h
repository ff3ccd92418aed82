// Device-side types and helpers of the attention kernels.
#pragma once

#include "attn_internal.h"
#include "qgemm_device.h"

namespace qg {

typedef __bf16 bf16;
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// An activation type: its pair conversion (round to nearest even) and its
// matrix instructions.
struct F16 {
  using T = f16;
  static constexpr float kLift = 11.0f, kSlack = 4.0f, kShrink = 0x1p-20f;   // of softmax weights, below
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const f32x2 x = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, f16x2));
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[0]; }
  static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[1]; }
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  // sum of a pair's values, and acc
  static __device__ __forceinline__ float add_pair(uint32_t w, float acc) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), f16x2{1, 1}, acc, false);
  }
  // two e4m3 codes (the low or high half of a word) as a pair; exact
  template <bool HIGH>
  static __device__ __forceinline__ uint32_t from_fp8(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
  }
};
struct BF16 {
  using T = bf16;
  static constexpr float kLift = 0.0f, kSlack = 8.0f, kShrink = 0.0f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const f32x2 x = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float add_pair(uint32_t w, float acc) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), bf16x2{1, 1}, acc, false);
  }
  template <bool HIGH>
  static __device__ __forceinline__ uint32_t from_fp8(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
  }
};

constexpr float kNegInf = -__builtin_huge_valf();
// Softmax weights are 2^(score - reference + lift) in the 16-bit type that meets the
// values (both in log2 units). The reference of a row moves only when a score passes
// it by the type's slack, so that the accumulators are rarely scaled; lift, a factor
// that the division by the sum of weights takes out again, puts the weights where the
// type has its bits:
//   bf16   lift 0, slack 8: no weight of a context of 2^24 tokens is too small for it.
//   fp16   lift 11, slack 4: weights end at 2^15, below the largest fp16 value. Those
//          above 2^-25 of the reference's keep all bits; a smaller one is off by up to
//          2^-36, and below that gone: the whole of 2^24 tokens loses at most 2^-12 of
//          the reference's weight. Without lift, a first token 18 nats above 20000
//          others took them nearly all away. At a slack of 8 the lift is at most 7 and
//          2^-32 the end, at the same speed (prefill of 4 prompts up to 2048 tokens,
//          32 heads: 104.7 us, here 105.2; every other case the same). The step from
//          2^15 to the type's end is one bit, and a score of 2^24 or more is itself off
//          by that much in fp32, so the slack shrinks with the reference, to none at
//          2^22: weights stay finite up to scores of 2^25.

// The score above which a row's reference moves.
template <class PF>
__device__ __forceinline__ float raise_limit(float mref) {
  if constexpr (PF::kShrink == 0.f) return mref + PF::kSlack;
  else return __builtin_fmaf(-PF::kShrink, fabsf(mref), mref + PF::kSlack);
}
// What a row's scores are taken from, by its reference.
template <class PF>
__device__ __forceinline__ float weight_base(float mref) {
  return mref == kNegInf ? 0.f : mref - PF::kLift;
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// A value at a wave-uniform address, through the scalar cache (data that no
// kernel writes while this one runs).
__device__ __forceinline__ int32_t scalar_load(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)p;
}
// n / d by a precomputed 1 / d, for 0 <= n < 2^31: (n + 1/2) / d is at least 1/(2d)
// away from every whole number, and its computed value off by less than 2^-20 / d.
__device__ __forceinline__ int divide(int n, double inverse) { return (int)(((double)n + 0.5) * inverse); }
__device__ __forceinline__ int divide_uniform(int n, double inverse) {
  return __builtin_amdgcn_readfirstlane(divide(n, inverse));
}
// Device-scope accesses of the parts' statistics.
__device__ __forceinline__ void store_shared(float* p, float x) {
  __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_shared(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Four outputs of a row: sums over its weight total; zeros where nothing was
// visible (a NaN total stays NaN).
template <class F>
__device__ __forceinline__ u32x2 finish(f32x4 o, float total, float v_scale) {
  const float f = v_scale / total;
  if (total == 0.f) return u32x2{0u, 0u};
  return u32x2{F::pack(o[0] * f, o[1] * f), F::pack(o[2] * f, o[3] * f)};
}

// Joins the parts of a row tile, in part order, and writes its outputs: row r of
// the tile to out + place(r). Called by every thread of the workgroup that arrived
// last, with 16 parts' loads in flight together (1 x 131072 tokens in 32 parts,
// e4m3: 46.9 us; 47.3 with 8 in flight, 59 with 32, which spill).
template <class F, class Place>
__device__ __forceinline__ void join_parts(const AttnArgs& p, int tile, int parts, int rows, const Place& place) {
  const int quads = p.head_dim / 4;
  const int64_t part_elems = (int64_t)p.part_rows * p.head_dim;
  const float* stats = p.stats + (int64_t)tile * p.splits * p.part_rows * 2;
  const float* partial = p.partial + (int64_t)tile * p.splits * part_elems;
  constexpr int kBatch = 16;   // parts whose loads are in flight together
  for (int x = threadIdx.x; x < rows * quads; x += blockDim.x) {
    const int row = x / quads, d = 4 * (x - row * quads);
    float m = kNegInf, total = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < parts; s0 += kBatch) {
      f32x4 y[kBatch];
      float ym[kBatch], yl[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int s = min(s0 + u, parts - 1);
        y[u] = load16_coherent(make_rsrc(partial + s * part_elems, (uint32_t)part_elems * 4),
                               (uint32_t)(row * p.head_dim + d) * 4);
        ym[u] = load_shared(stats + ((int64_t)s * p.part_rows + row) * 2);
        yl[u] = load_shared(stats + ((int64_t)s * p.part_rows + row) * 2 + 1);
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) top = fmaxf(top, ym[u]);   // re-read last parts change nothing
      const float base = top == kNegInf ? 0.f : top;
      const float f0 = exp2_of(m - base);
      total *= f0;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= f0;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (s0 + u < parts) {
          const float f = exp2_of(ym[u] - base);
          total += f * yl[u];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] += f * y[u][i];
        }
      }
      m = top;
    }
    typename F::T* dst = static_cast<typename F::T*>(p.out) + place(row) + d;
    *reinterpret_cast<u32x2*>(dst) = finish<F>(o, total, p.v_scale);
  }
}

// Bytes picked from a (selectors 0-3) and b (4-7).
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b, uint32_t sel) {
  return __builtin_amdgcn_perm(b, a, sel);
}
constexpr uint32_t kLows = 0x05040100u;    // low halves of a and b
constexpr uint32_t kHighs = 0x07060302u;   // high halves of a and b

// The tokens that one query position sees: j <= last and (j >= low or j < sinks).
// Whole blocks between the last sink block and the first window block are
// skipped: virtual block v stands for block v, or v + skip past the sink blocks.
struct Visible {
  int len;          // tokens 0..len-1 exist
  int low;          // first token of the window
  int sinks;        // visible tokens before it
  int sink_blocks;
  int skip;
  int blocks;       // virtual blocks
  __device__ __forceinline__ Visible(int len_, int low_, int sinks_) {
    len = len_;
    low = max(0, low_);
    sinks = min(sinks_, low);
    sink_blocks = (sinks + kTokBlock - 1) / kTokBlock;
    skip = max(0, low / kTokBlock - sink_blocks);
    blocks = (len + kTokBlock - 1) / kTokBlock - skip;
  }
  __device__ __forceinline__ int block(int v) const { return v < sink_blocks ? v : v + skip; }
  __device__ __forceinline__ bool whole(int blk) const {   // every token of the block is visible
    const int j0 = blk * kTokBlock;
    return j0 + kTokBlock <= len && (j0 >= low || j0 + kTokBlock <= sinks);
  }
  __device__ __forceinline__ bool sees(int j) const { return j < len && (j >= low || j < sinks); }
};

// Page of a token block and the element offset of the block's first token in it.
__device__ __forceinline__ int page_of(const CacheArgs& c, int blk, int* place) {
  const int col = c.magic ? (int)__umulhi((uint32_t)blk, c.magic) : blk;
  *place = blk - col * c.page_blocks;
  return col;
}

}  // namespace qg
