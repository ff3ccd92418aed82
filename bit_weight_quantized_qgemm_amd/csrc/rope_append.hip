// Norms of queries and keys per head, position rotation and the store of keys
// and values into the paged cache, in one pass:
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin).
//
// A head is 16 values per lane over 4, 8 or 16 lanes (head_dim up to 64, 128,
// 256); the sum of squares is joined by cross-lane adds. A lane holds eight
// whole rotation pairs: 8 consecutive values of the first half and the 8 that
// pair with them (or 16 consecutive values of interleaved pairs), so the
// rotation needs no exchange and every access is 16 bytes. The values past
// rot_dim are paired the same way and pass through.
//
// The op reads each head once and writes it once. 8192 tokens of 64/8 heads of 128,
// bf16, take 64 us (336 MB, 5.2 TB/s; a large copy reaches 4.9); 1003 tokens of
// 32/32 heads of 80 9.5 us, where most of the time is the chain launch, position,
// table entry, store; one token 3.7 us, the launch. A lane takes 16 values, not 8,
// because the pairs of the split rotation then meet in one lane without an exchange.
#include "attn_device.h"

namespace qg {
namespace {

// Eight values as four words.
template <class F>
__device__ __forceinline__ void unpack8(u32x4 w, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = F::lo(w[i]);
    x[2 * i + 1] = F::hi(w[i]);
  }
}
template <class F>
__device__ __forceinline__ u32x4 pack8(const float* x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = F::pack(x[2 * i], x[2 * i + 1]);
  return w;
}
// Saturated e4m3 codes; NaN stays NaN (the clamp alone would turn it into a number).
__device__ __forceinline__ float clamp_fp8(float x) { return x != x ? x : fminf(fmaxf(x, -448.f), 448.f); }
__device__ __forceinline__ u32x2 pack8_fp8(const float* x, float scale) {
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_fp8(x[4 * i] / scale), clamp_fp8(x[4 * i + 1] / scale), 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_fp8(x[4 * i + 2] / scale), clamp_fp8(x[4 * i + 3] / scale), p, true);
    w[i] = (uint32_t)p;
  }
  return w;
}

template <class F, bool FP8, bool INTERLEAVED, int LANES>
__global__ void __launch_bounds__(256) rope_append(AppendArgs p) {
  using T = typename F::T;
  constexpr int kHeads = 256 / LANES;   // heads of a workgroup
  const int lane = threadIdx.x % LANES;
  const int heads = p.q_heads + 2 * p.kv_heads;
  // below 2^31, or in the last workgroup a little above, which wraps to a negative
  const int task = (int)((blockIdx.x + p.first_block) * (uint32_t)kHeads + threadIdx.x / LANES);
  const int token = divide(task, p.inv_heads);
  if (task < 0 || token >= p.num_tokens) return;   // whole heads of lanes leave together
  int head = task - token * heads;
  const bool live = lane * 16 < p.head_dim;

  const int pos = p.positions[token];
  const bool padding = pos < 0 || pos >= p.rope_rows;
  enum { Q, K, V };
  const int what = head < p.q_heads ? Q : head < p.q_heads + p.kv_heads ? K : V;
  if (padding && what != Q) return;

  // places of the lane's two runs of eight values
  const int half = p.rot_dim / 2;
  int ia, ib;
  bool turned;
  if (INTERLEAVED || what == V) {
    ia = 16 * lane;
    ib = ia + 8;
    turned = ia < p.rot_dim;
  } else {
    turned = 8 * lane < half;
    ia = turned ? 8 * lane : p.rot_dim + 8 * lane - half;
    ib = ia + (turned ? half : (p.head_dim - p.rot_dim) / 2);
  }
  const T* src;
  if (what == Q) {
    src = static_cast<const T*>(p.q) + token * p.q_ts + head * p.q_hs;
  } else if (what == K) {
    head -= p.q_heads;
    src = static_cast<const T*>(p.k) + token * p.k_ts + head * p.k_hs;
  } else {
    head -= p.q_heads + p.kv_heads;
    src = static_cast<const T*>(p.v) + token * p.v_ts + head * p.v_hs;
  }
  u32x4 wa = {0, 0, 0, 0}, wb = {0, 0, 0, 0};
  if (live) {
    wa = *reinterpret_cast<const u32x4*>(src + ia);
    wb = *reinterpret_cast<const u32x4*>(src + ib);
  }
  // where a key or value goes, looked up while the head itself is on its way
  int page = -1, place = 0;
  if (what != Q) {
    const int seq = p.token_seq ? p.token_seq[token] : token;
    const int col = page_of(p.cache, pos / kTokBlock, &place);
    if (seq >= 0 && seq < p.num_seqs && col < p.cache.table_stride) page = p.cache.table[seq * p.cache.table_stride + col];
  }
  float a[8], b[8];
  unpack8<F>(wa, a);
  unpack8<F>(wb, b);

  const T* norm = static_cast<const T*>(what == Q ? p.q_norm : what == K ? p.k_norm : nullptr);
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += a[i] * a[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += b[i] * b[i];
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (live) {
      const float r = 1.0f / sqrtf(sum * p.inv_dim + p.eps);
      float w[8];
      unpack8<F>(*reinterpret_cast<const u32x4*>(norm + ia), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = a[i] * r * w[i];
      unpack8<F>(*reinterpret_cast<const u32x4*>(norm + ib), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = b[i] * r * w[i];
    }
  }
  if (!live) return;
  if (what != V && turned && !padding) {
    const float* row = p.rope + (int64_t)pos * p.rot_dim;
    const f32x4* cs = reinterpret_cast<const f32x4*>(row + 8 * lane);
    const f32x4* sn = reinterpret_cast<const f32x4*>(row + half + 8 * lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = cs[i / 4][i % 4], s = sn[i / 4][i % 4];
      float& x = INTERLEAVED ? (i < 4 ? a[2 * (i % 4)] : b[2 * (i % 4)]) : a[i];
      float& y = INTERLEAVED ? (i < 4 ? a[2 * (i % 4) + 1] : b[2 * (i % 4) + 1]) : b[i];
      const float xr = x * c - y * s;
      y = y * c + x * s;
      x = xr;
    }
  }

  if (what == Q) {
    T* dst = static_cast<T*>(p.q_out) + token * p.qo_ts + head * p.qo_hs;
    const u32x4 zero = {0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(dst + ia) = padding ? zero : pack8<F>(a);
    *reinterpret_cast<u32x4*>(dst + ib) = padding ? zero : pack8<F>(b);
    return;
  }
  if (page < 0 || page >= p.cache.num_pages) return;
  const int64_t at = page * p.cache.page_stride + (place * kTokBlock + pos % kTokBlock) * p.cache.token_stride +
                     head * p.cache.head_stride;
  void* base = const_cast<void*>(what == K ? p.cache.k : p.cache.v);
  if (FP8) {
    const float scale = what == K ? p.k_scale : p.v_scale;
    uint8_t* dst = static_cast<uint8_t*>(base) + at;
    *reinterpret_cast<u32x2*>(dst + ia) = pack8_fp8(a, scale);
    *reinterpret_cast<u32x2*>(dst + ib) = pack8_fp8(b, scale);
  } else {
    T* dst = static_cast<T*>(base) + at;
    *reinterpret_cast<u32x4*>(dst + ia) = pack8<F>(a);
    *reinterpret_cast<u32x4*>(dst + ib) = pack8<F>(b);
  }
}

template <class F, bool FP8, bool INTERLEAVED>
hipError_t launch_lanes(const AppendArgs& a, hipStream_t s) {
  const int lanes = a.head_dim <= 64 ? 4 : a.head_dim <= 128 ? 8 : 16;
  const int64_t tasks = (int64_t)a.num_tokens * (a.q_heads + 2 * a.kv_heads);
  return launch_in_runs((tasks * lanes + 255) / 256, [&](dim3 grid, uint32_t first) {
    AppendArgs r = a;
    r.first_block = first;
    switch (lanes) {
      case 4: hipLaunchKernelGGL((rope_append<F, FP8, INTERLEAVED, 4>), grid, dim3(256), 0, s, r); break;
      case 8: hipLaunchKernelGGL((rope_append<F, FP8, INTERLEAVED, 8>), grid, dim3(256), 0, s, r); break;
      default: hipLaunchKernelGGL((rope_append<F, FP8, INTERLEAVED, 16>), grid, dim3(256), 0, s, r); break;
    }
  });
}

template <class F>
hipError_t launch_type(const AppendArgs& a, bool fp8, bool interleaved, hipStream_t s) {
  if (fp8) return interleaved ? launch_lanes<F, true, true>(a, s) : launch_lanes<F, true, false>(a, s);
  return interleaved ? launch_lanes<F, false, true>(a, s) : launch_lanes<F, false, false>(a, s);
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, bool bf16, bool fp8, bool interleaved, hipStream_t s) {
  return bf16 ? launch_type<BF16>(a, fp8, interleaved, s) : launch_type<F16>(a, fp8, interleaved, s);
}

}  // namespace qg
