// Internal interface between the host code of the dense operators
// (moe_dense_api.cpp) and their gfx950 kernels (moe_norm_kernels.hip,
// moe_gated_kernels.hip, moe_adapter_kernels.hip).  Not
// installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "moe_ep.h"
#include "moe_tile_rule.h"

namespace moe_ep_detail {

struct NormKArgs {
  const uint16_t* x;
  const uint16_t* residual;   // or NULL
  const void* weight;
  void* out;
  float* scales;              // 8-bit rows only
  uint16_t* residual_out;     // or NULL
  int64_t x_stride, residual_stride, out_stride, scales_stride, residual_out_stride;
  int32_t n;
  int32_t hidden;
  int32_t group;              // 8-bit rows: columns of a scale; 0: a whole row
  float eps;
};

// One operand of a matrix product: element (row, k) is p[row * stride + k], or
// p[k * stride + row] where the rows lie side by side.
struct MatK {
  const uint16_t* p;
  int64_t stride;
  int32_t rows;               // of a gated weight: of each half
  // Whether tiles may be loaded in whole 16-byte units: base, stride and the
  // side by side extent are multiples of them, and the stride is at most 2^22
  // (offsets inside a tile have 32 bits).
  bool whole;
};

struct GatedKArgs {
  MatK w, x;
  int32_t hidden;
  int32_t inter;
  void* out;                  // [n, inter]
  float* pre;                 // [n, 2 * inter] gate and up, or NULL
  int64_t out_stride;
  int32_t out_f32;
  int32_t ptiles, qtiles;     // (set by the launcher)
};

// out[q][p] = *factor * sum over k of (q + q_rest) p
struct ProductKArgs {
  MatK p, q;
  int32_t k;
  int32_t q_rows;             // rows of out (q may have more, of no account)
  uint16_t* out;
  int64_t out_stride;
  const float* factor;        // or NULL: 1
  // Elements from q to what q lacks (float16: times kRestUpF16), which lies as
  // q does; or 0.
  int64_t q_rest;
  float* partial;             // kPartialFloats: sums over parts of k, where there are few results
  int32_t ptiles, qtiles;     // (set by the launcher)
  int32_t parts;              // (set by the launcher)
};

// d = [dgate, dup] of a gated product, times a power of two for float16.
struct GatedGradKArgs {
  const void* dout;           // [n, inter]
  const float* pre;           // [n, 2 * inter]
  uint16_t* d;                // [n, d_stride], columns from 2 * inter on are not written
  uint16_t* rest;             // or NULL: what d's rounding leaves (float16: times kRestUpF16), as d lies
  int64_t dout_stride, d_stride;
  int32_t dout_f32;
  int32_t n, inter;
  uint32_t* tops;             // float16: [kTops] largest magnitudes
  float* factor;              // float16: what the products are multiplied with
};
constexpr int kTops = 1024;
// float16 keeps what a rounding leaves (2^-11 of the number at most) times
// 2^11, so that its smallest values are not lost.
constexpr float kRestUpF16 = 2048.0f;

struct AdapterKArgs {
  MatK w, x;
  int32_t k;
  void* out;                  // [n, out_features]
  int64_t out_stride;
  int32_t out_f32;
  const uint16_t* a;          // [adapters, rank, in_features]
  void* low;                  // scale * A x of each row with its adapter: LowSpace
  int32_t low_stride;
  const uint16_t* b;          // [adapters, out_features, rank]
  const int32_t* ids;         // [n]
  const float* scales;        // [adapters] or NULL
  int32_t adapters, rank;
  int32_t ptiles, qtiles;     // (set by the launcher)
};

// dtype: MOE_EP_BF16 or MOE_EP_F16.
hipError_t launch_gated(const GatedKArgs& a, int dtype, hipStream_t stream);
hipError_t launch_gated_grad(const GatedGradKArgs& a, int dtype, hipStream_t stream);
// p lies with its rows side by side; q with its rows side by side, or with k (q_kc).
hipError_t launch_product(const ProductKArgs& a, int dtype, bool q_kc, hipStream_t stream);
// The low-rank values between the two kernels, zeros from the rank to the
// stride.  Few rows: float32 [kLowSplits, rows, stride], sums over parts of k.
// Else their bfloat16 parts [kParts, rows, stride].
constexpr int kLowFew = 64, kLowSplits = 4;
struct LowSpace {
  int32_t stride;
  int64_t bytes;
  LowSpace(int64_t rows, int32_t rank) {
    const bool few = rows <= kLowFew;
    stride = few ? (rank + 7) / 8 * 8 : (rank + 31) / 32 * 32;
    bytes = rows * stride * (few ? 4 * kLowSplits : 2 * 3);
  }
};
hipError_t launch_adapter(const AdapterKArgs& a, int dtype, hipStream_t stream);
hipError_t launch_rms_norm(const NormKArgs& a, int dtype, bool weight_f32, bool eight, hipStream_t stream);

}  // namespace moe_ep_detail
