// Device types that the expert-side kernels share: the 16-bit element types
// with their matrix instruction, conversions and 4-bit decode.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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
  // v as high + low: 16 significant bits.  Infinities and NaN stay in the high part.
  static __device__ __forceinline__ void split(float v, uint16_t* hi, uint16_t* lo) {
    *hi = from_float(v);
    const float h = to_float(*hi);
    *lo = __builtin_isfinite(h) ? from_float(v - h) : (uint16_t)0;
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
  // 22 significant bits up to 65504; a finite value beyond that keeps the
  // rest in the low part, and saturates at 131008.
  static __device__ __forceinline__ void split(float v, uint16_t* hi, uint16_t* lo) {
    if (!__builtin_isfinite(v)) {
      *hi = from_float(v);
      *lo = 0;
      return;
    }
    *hi = from_float(__builtin_fminf(__builtin_fmaxf(v, -65504.0f), 65504.0f));
    *lo = from_float(__builtin_fminf(__builtin_fmaxf(v - to_float(*hi), -65504.0f), 65504.0f));
  }
};

}  // namespace
}  // namespace moe_ep_detail
