// Argument checks that the host code of the operators over rows shares
// (moe_experts_api.cpp, moe_dense_api.cpp).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "moe_ep.h"

namespace moe_ep_detail {

// Records a failed call's message for moe_ep_last_error() and returns status
// (moe_ep_api.cpp).
int report(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline int elem_bytes(int dtype) {
  switch (dtype) {
    case MOE_EP_F32: return 4;
    case MOE_EP_BF16: return 2;
    case MOE_EP_F16: return 2;
    default: return 0;
  }
}

inline int64_t up(int64_t x, int64_t a) {
  return (x + a - 1) / a * a;
}

// The kernels run on the current device's memory: a stream of another device
// is refused.
inline int check_stream(void* stream) {
  if (!stream) return MOE_EP_OK;
  int cur = -1, dev = -1;
  if (hipGetDevice(&cur) != hipSuccess || hipStreamGetDevice(static_cast<hipStream_t>(stream), &dev) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_EP_OK;
  }
  if (cur != dev)
    return report(MOE_EP_ERR_INVALID_ARG, "the stream runs on device %d but the current device is %d", dev, cur);
  return MOE_EP_OK;
}

inline int check_rows(const char* what, const void* p, int64_t stride, int64_t width, int n, int esz, bool repeat) {
  if (stride < 0 || (n > 1 && stride < width && !(repeat && stride == 0)) || stride > INT64_MAX / 8 / std::max(n, 1))
    return report(MOE_EP_ERR_INVALID_ARG, "%s: row stride %lld with rows of %lld", what, (long long)stride,
                  (long long)width);
  if (n > 0 && !p) return report(MOE_EP_ERR_INVALID_ARG, "%s is NULL with %d rows", what, n);
  if (!aligned_to(p, esz)) return report(MOE_EP_ERR_ALIGN, "%s not aligned to its element", what);
  return MOE_EP_OK;
}

// Whether the byte ranges from the first to the last element of two row sets meet.
inline bool overlap(const void* a, int64_t a_stride, int64_t a_width, int a_esz, const void* b, int64_t b_stride,
             int64_t b_width, int b_esz, int n) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + (uintptr_t)(((n - 1) * a_stride + a_width) * a_esz);
  const uintptr_t b1 = b0 + (uintptr_t)(((n - 1) * b_stride + b_width) * b_esz);
  return a0 < b1 && b0 < a1;
}

inline int check_types(int dtype, int out_dtype) {
  if (dtype != MOE_EP_BF16 && dtype != MOE_EP_F16)
    return report(MOE_EP_ERR_INVALID_ARG, "dtype %d is not MOE_EP_BF16 or MOE_EP_F16", dtype);
  if (out_dtype != dtype && out_dtype != MOE_EP_F32)
    return report(MOE_EP_ERR_INVALID_ARG, "out_dtype %d is neither dtype %d nor MOE_EP_F32", out_dtype, dtype);
  return MOE_EP_OK;
}

// Largest matrix side: row and column indexes (and two rows of tiles past
// them) are 32-bit in the kernels, offsets 64-bit, and a launch has fewer than
// 2^32 threads in x (down_kernel: 512 for 16 columns and 128 of 2048 tokens).
constexpr int32_t kMaxSide = 1 << 22;
// Fewest elements of a row that the kernels read eight at a time.
constexpr int32_t kMinRow = 8;

}  // namespace moe_ep_detail
