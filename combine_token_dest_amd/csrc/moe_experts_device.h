// Device types that the expert-side kernels share: the 16-bit element types
// with their matrix instruction, conversions and 4-bit decode.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_experts_internal.h"

namespace moe_ep_detail {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct BF16 {
  static __device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t nibbles(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, HI));
  }
  static constexpr uint32_t kMinus8 = 0xC100C100u;   // two of -8.0
  static __device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t from_float(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
  }
};

struct F16 {
  static __device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t nibbles(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 512.0f, HI));
  }
  static constexpr uint32_t kMinus8 = 0xC800C800u;
  static __device__ __forceinline__ float to_float(uint16_t v) {
    return static_cast<float>(__builtin_bit_cast(_Float16, v));
  }
  static __device__ __forceinline__ uint16_t from_float(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
  }
};

// v as the sum of kParts bfloat16 (moe_experts_internal.h): 8 significant bits
// cut off after another, so that nothing is rounded: the three hold float32's
// 24 bits in float32's range (below 2^-110 the last ones end at bfloat16's
// smallest value).  An infinity or NaN stays in the first.
__device__ __forceinline__ void split_parts(float v, uint16_t (&part)[kParts]) {
  const bool finite = __builtin_isfinite(v);
  const uint32_t u0 = __float_as_uint(v);
  const float r1 = v - __uint_as_float(u0 & 0xFFFF0000u);
  const uint32_t u1 = __float_as_uint(r1);
  const uint32_t u2 = __float_as_uint(r1 - __uint_as_float(u1 & 0xFFFF0000u));
  part[0] = finite ? (uint16_t)(u0 >> 16) : BF16::from_float(v);
  part[1] = finite ? (uint16_t)(u1 >> 16) : (uint16_t)0;
  part[2] = finite ? (uint16_t)(u2 >> 16) : (uint16_t)0;
}

// Eight floats as their parts.
__device__ __forceinline__ void split_floats(const u32x4 (&v)[2], u32x4 (&part)[kParts]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u[2][kParts];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float x = __uint_as_float(v[i >> 1][(i & 1) * 2 + c]);
      u[c][0] = __float_as_uint(x);
      float r = x - __uint_as_float(u[c][0] & 0xFFFF0000u);
      r = r == r ? r : 0.0f;              // of an infinity
      u[c][1] = __float_as_uint(r);
      u[c][2] = __float_as_uint(r - __uint_as_float(u[c][1] & 0xFFFF0000u));
    }
#pragma unroll
    for (int pl = 0; pl < kParts; ++pl) part[pl][i] = u[0][pl] >> 16 | (u[1][pl] & 0xFFFF0000u);
  }
}

// Eight float16 as the sums of two bfloat16 each: 8 bits, then the other 3.
// Exact for finite values.
__device__ __forceinline__ void split_f16(const u32x4& v, u32x4* hi, u32x4* lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = F16::to_float((uint16_t)v[i]), b = F16::to_float((uint16_t)(v[i] >> 16));
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b) & 0xFFFF0000u;
    const float ra = a - __uint_as_float(ua & 0xFFFF0000u), rb = b - __uint_as_float(ub);
    (*hi)[i] = ua >> 16 | ub;
    (*lo)[i] = __float_as_uint(ra) >> 16 | (__float_as_uint(rb) & 0xFFFF0000u);
  }
}

}  // namespace
}  // namespace moe_ep_detail
