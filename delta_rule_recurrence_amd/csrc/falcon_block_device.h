// Device-side helpers of the operators around the recurrence (gfx950, wave64).
#pragma once

#include "falcon_block.h"
#include "falcon_device.h"

namespace falcon {

// ---- V consecutive elements as floats ----------------------------------------
// V is one, or a multiple of four: wide accesses of 16 bytes (8 for four bf16), the
// address a multiple of that.
template <typename IO, int V>
__device__ __forceinline__ void load_vec(const IO* p, float (&out)[V]) {
  static_assert(V == 1 || V % 4 == 0);
  static_assert(sizeof(IO) == 4 || V == 1 || V == 4 || V % 8 == 0);
  if constexpr (V == 1) {
    out[0] = io<IO>::load(p, 0);
  } else if constexpr (sizeof(IO) == 2) {
    if constexpr (V % 8 == 0) {
#pragma unroll
      for (int k = 0; k < V / 8; ++k) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[k];
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          out[8 * k + 2 * i] = __uint_as_float(w[i] << 16);
          out[8 * k + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      out[0] = __uint_as_float(a.x << 16);
      out[1] = __uint_as_float(a.x & 0xffff0000u);
      out[2] = __uint_as_float(a.y << 16);
      out[3] = __uint_as_float(a.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      const float4 a = reinterpret_cast<const float4*>(p)[k];
      out[4 * k] = a.x;
      out[4 * k + 1] = a.y;
      out[4 * k + 2] = a.z;
      out[4 * k + 3] = a.w;
    }
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return static_cast<uint32_t>(f32_to_bf16(lo)) | (static_cast<uint32_t>(f32_to_bf16(hi)) << 16);
}

// Results are rounded once, to the I/O type, as they are stored.
template <typename IO, int V>
__device__ __forceinline__ void store_vec(IO* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    io<IO>::store(p, 0, v[0]);
  } else if constexpr (sizeof(IO) == 2) {
    if constexpr (V % 8 == 0) {
#pragma unroll
      for (int k = 0; k < V / 8; ++k)
        reinterpret_cast<uint4*>(p)[k] = make_uint4(bf16_pair(v[8 * k], v[8 * k + 1]), bf16_pair(v[8 * k + 2], v[8 * k + 3]),
                                                    bf16_pair(v[8 * k + 4], v[8 * k + 5]), bf16_pair(v[8 * k + 6], v[8 * k + 7]));
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < V / 4; ++k)
      reinterpret_cast<float4*>(p)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  }
}

// ---- activations ----------------------------------------------------------------
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp_f32(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// f(p) and f'(p).
template <int ACT>
__device__ __forceinline__ float act_f32(float p) {
  if constexpr (ACT == kActSilu) return p * sigmoid_f32(p);
  if constexpr (ACT == kActElu1) return p > 0.0f ? p + 1.0f : exp_f32(p);
  if constexpr (ACT == kActSigmoid) return sigmoid_f32(p);
  return p;
}
template <int ACT>
__device__ __forceinline__ float act_slope_f32(float p) {
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid_f32(p);
    return s * (1.0f + p * (1.0f - s));
  }
  if constexpr (ACT == kActElu1) return p > 0.0f ? 1.0f : exp_f32(p);
  if constexpr (ACT == kActSigmoid) {
    const float s = sigmoid_f32(p);
    return s * (1.0f - s);
  }
  return 1.0f;
}

// log(1 + exp(v)) = max(v, 0) + log1p(u), u = exp(-|v|).  1 + u rounds to w;
// what the rounding lost, u - (w - 1), is exact and returns as its first-order
// term, so small steps keep their relative accuracy.
__device__ __forceinline__ float softplus_f32(float v) {
  const float u = exp_f32(-fabsf(v));
  const float w = 1.0f + u;
  const float lost = u - (w - 1.0f);
  return fmaxf(v, 0.0f) + __builtin_fmaf(__builtin_amdgcn_logf(w), kLn2, lost * __builtin_amdgcn_rcpf(w));
}

// ---- sums over lanes ---------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_plus(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// Sum over aligned groups of LANES (a power of two up to 64) lanes, in every
// lane; the whole wave must be active.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LANES >= 2) v = dpp_plus<0xb1>(v);    // quad_perm [1, 0, 3, 2]
  if constexpr (LANES >= 4) v = dpp_plus<0x4e>(v);    // quad_perm [2, 3, 0, 1]
  if constexpr (LANES >= 8) v = dpp_plus<0x141>(v);   // row_half_mirror
  if constexpr (LANES >= 16) v = dpp_plus<0x140>(v);  // row_mirror
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
  if constexpr (LANES >= 64) v += __shfl_xor(v, 32);
  return v;
}

// Workgroups b, b + 8, b + 16, ... run on one XCD: this order lets neighbours, which
// share cache lines or rows, follow one another there.
__device__ __forceinline__ int64_t by_xcd(int64_t block, int64_t blocks) {
  const int64_t each = blocks / 8, more = blocks % 8, x = block % 8;
  return x * each + min(x, more) + block / 8;
}

// Tokens of sequence b, between 0 and T.
__device__ __forceinline__ int tokens_of(const int32_t* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace falcon
