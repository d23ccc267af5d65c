// Rows of logits in registers: what the kernels share that take a tempered, masked
// softmax of a row (token log-probabilities, distillation and their gradients).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_device.hpp"

namespace qs {
namespace score {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// |k_w| up to which exponents may be taken against k_w: its rounding, the exponent
// of the sums' common factor, is at most 1/2 there
constexpr float kFused = 16777216.0f;

template <int DT> constexpr int kPer = DT == QS_F32 ? 4 : 8;  // tokens per 16-byte load

// log2(e) / T held to finite, non-zero values: 0 times it is 0, and -inf
// times it is -inf. (Past T = 1.2e38 it is below the least normal float32, still
// good to 2^-22 of itself.)
__device__ __forceinline__ float scale_of(float T) {
  return fminf(fmaxf(kLog2e / T, 1.4e-45f), 3.4e38f);
}

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}
__device__ __forceinline__ float readlane_f32(float v, int l) {
  return __uint_as_float(readlane_u32(__float_as_uint(v), l));
}
__device__ __forceinline__ float wave_max_f32(float v) {
  v = fmaxf(v, dpp_f32<kDppXor1>(v));
  v = fmaxf(v, dpp_f32<kDppXor2>(v));
  v = fmaxf(v, dpp_f32<kDppHalfMirror>(v));
  v = fmaxf(v, dpp_f32<kDppMirror>(v));
  return fmaxf(fmaxf(readlane_f32(v, 0), readlane_f32(v, 16)),
               fmaxf(readlane_f32(v, 32), readlane_f32(v, 48)));
}
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += dpp_f32<kDppXor1>(v);
  v += dpp_f32<kDppXor2>(v);
  v += dpp_f32<kDppHalfMirror>(v);
  v += dpp_f32<kDppMirror>(v);
  return (readlane_f32(v, 0) + readlane_f32(v, 16)) + (readlane_f32(v, 32) + readlane_f32(v, 48));
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// f_w of the join; exponents below -200 weigh nothing against the maximum's 1.
__device__ __forceinline__ float rel(float m, float top, float c) {
  return fmaxf((m - top) * c, -200.0f);
}

// Token e (0 .. kPer - 1) of a 16-byte load, as float.
template <int DT>
__device__ __forceinline__ float token(const uint4& v, int e) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (DT == QS_F32) return __uint_as_float(w[e]);
  return __uint_as_float((e & 1) ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16));
}

template <int DT>
__device__ __forceinline__ float logit_at(const uint8_t* row, int i) {
  if constexpr (DT == QS_F32) return reinterpret_cast<const float*>(row)[i];
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
}

// Masks of a 16-byte load's registers: all ones where the token's bit is set.
template <int DT>
__device__ __forceinline__ uint4 masks_of(uint32_t bits) {
  uint32_t w[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if constexpr (DT == QS_F32) {
      w[d] = (uint32_t)__builtin_amdgcn_sbfe((int)bits, d, 1);
    } else {
      const uint32_t lo = (uint32_t)__builtin_amdgcn_sbfe((int)bits, 2 * d, 1);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_sbfe((int)bits, 2 * d + 1, 1);
      w[d] = bfi(0xFFFFu, lo, hi);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Tokens outside the masks become -inf.
template <int DT>
__device__ __forceinline__ uint4 blank(const uint4& v, const uint4& keep) {
  constexpr uint32_t kFill = DT == QS_F32 ? 0xFF800000u : 0xFF80FF80u;
  return make_uint4(bfi(keep.x, v.x, kFill), bfi(keep.y, v.y, kFill), bfi(keep.z, v.z, kFill),
                    bfi(keep.w, v.w, kFill));
}
// The largest of the tokens a lane has seen. bf16 tokens are compared two at a
// time as whole numbers: among those with a clear sign the larger signed number
// is the larger token, among the others the smaller unsigned one.
template <int DT> struct Largest;
template <> struct Largest<QS_F32> {
  float m = -INFINITY;
  __device__ __forceinline__ void add(const uint4& v) {
    m = fmaxf(fmaxf(m, __uint_as_float(v.x)), __uint_as_float(v.y));
    m = fmaxf(fmaxf(m, __uint_as_float(v.z)), __uint_as_float(v.w));
  }
  __device__ __forceinline__ float value() const { return m; }
};
template <> struct Largest<QS_BF16> {
  uint32_t above = 0x80008000u, below = 0xFFFFFFFFu;
  __device__ __forceinline__ void add(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      above = bits_of(__builtin_elementwise_max(as_s2(above), as_s2(w[d])));
      below = bits_of(__builtin_elementwise_min(as_u2(below), as_u2(w[d])));
    }
  }
  __device__ __forceinline__ float value() const {
    const int hi = max((int)above >> 16, (int)(above << 16) >> 16);
    const uint32_t lo = min(below >> 16, below & 0xFFFFu);
    return __uint_as_float((hi >= 0 ? (uint32_t)hi : lo) << 16);
  }
};

// Keeps the compiler from holding a load's unpacked tokens from one pass over
// the registers to the next (unpacking again costs less than the registers).
__device__ __forceinline__ void opaque(uint4& v) {
  asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));
}

}  // namespace
}  // namespace score
}  // namespace qs
