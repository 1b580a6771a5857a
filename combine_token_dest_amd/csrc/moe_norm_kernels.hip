// gfx950 kernel of the root-mean-square norm with the residual's addition:
// s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, the rows leaving
// in 16 bits or as e4m3 with a scale for each group of columns.
//
// One read of x and residual and one write of each output is all it has to
// move (8-bit rows with a residual: 7 bytes a column), so it is bound by HBM: a
// copy of 2 GiB runs at 4.9 TB/s, 8192 rows of 4096 in 16 bits at 5.8 (46 us)
// and 4096 of 7168 with a residual to 8 bits at 4.6 (45 us).  A workgroup takes one row and keeps s in registers
// between the sum of squares and the outputs; the squares are summed in
// float64, which hides behind the loads and cannot overflow.
//
// Maxima of magnitudes are taken over the bits as integers: NaN is above
// infinity there, so it is not lost, as it would be in a float maximum.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "moe_dense_internal.h"
#include "moe_experts_device.h"

namespace moe_ep_detail {
namespace {

// 16-byte (and 8-byte) accesses from any element address.
struct __attribute__((packed, aligned(2))) Half8 {
  u32x4 v;
};
struct __attribute__((packed, aligned(4))) Float4 {
  f32x4 v;
};
struct __attribute__((packed, aligned(1))) Byte8 {
  u32x2 v;
};

// Elements c .. c + 7 of a row as floats; those past `have` are 0.
template <class T>
__device__ __forceinline__ void load_row8(const uint16_t* p, int have, float (&v)[8]) {
  if (have >= 8) {
    const u32x4 w = reinterpret_cast<const Half8*>(p)->v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = T::to_float((uint16_t)w[e]);
      v[2 * e + 1] = T::to_float((uint16_t)(w[e] >> 16));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < have ? T::to_float(p[e]) : 0.0f;
  }
}
__device__ __forceinline__ void load_row8(const float* p, int have, float (&v)[8]) {
  if (have >= 8) {
    const f32x4 a = reinterpret_cast<const Float4*>(p)->v, b = reinterpret_cast<const Float4*>(p + 4)->v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[e + 4] = b[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < have ? p[e] : 0.0f;
  }
}

template <class T>
__device__ __forceinline__ void store_row8(uint16_t* p, int have, const float (&v)[8]) {
  if (have >= 8) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = (uint32_t)T::from_float(v[2 * e]) | (uint32_t)T::from_float(v[2 * e + 1]) << 16;
    reinterpret_cast<Half8*>(p)->v = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < have) p[e] = T::from_float(v[e]);
  }
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Rounds eight values to e4m3 (to nearest even; NaN stays NaN).  They are at
// most 448 but for the last bits of a quotient, which are rounded away.
__device__ __forceinline__ void store_e4m3(uint8_t* p, int have, const float (&q)[8]) {
  u32x2 w = {0, 0};
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    w[e >> 1] = __builtin_amdgcn_cvt_pk_fp8_f32(q[2 * e], q[2 * e + 1], w[e >> 1], false);
    w[e >> 1] = __builtin_amdgcn_cvt_pk_fp8_f32(q[2 * e + 2], q[2 * e + 3], w[e >> 1], true);
  }
  if (have >= 8) {
    reinterpret_cast<Byte8*>(p)->v = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < have) p[e] = (uint8_t)(w[e >> 2] >> (e & 3) * 8);
  }
}

// 448 v / top of a group with the largest magnitude top, whose scale is
// m top / 448.  The factor 448 / top has two parts, so beside v's own roundings
// only the quotient's is left: every other one would put more quotients on the
// wrong side of the middle between two e4m3 values.  A scale near float32's end
// may be rounded by any share, so there it is what is divided by, brought up by
// 2^100 as v is, and the quotient needs an end.
__device__ __forceinline__ void divide(float (&v)[8], float top, float scale, float m) {
  if (scale < 0x1p-64f) {
    const float inv = scale == 0.0f ? 0.0f : m / (scale * 0x1p100f);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fminf(fmaxf(v[e] * 0x1p100f * inv, -448.0f), 448.0f);
  } else {
    const float high = 448.0f / top;                       // 0 of an infinity, NaN of NaN
    const float low = high > 0.0f ? __builtin_fmaf(-top, high, 448.0f) / top : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(v[e], high, v[e] * low);
  }
}

// Sum and maximum over a workgroup, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* part, int waves) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = part[0];
  for (int w = 1; w < waves; ++w) sum += part[w];
  return sum;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* part, int waves) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t top = part[0];
  for (int w = 1; w < waves; ++w) top = max(top, part[w]);
  return top;
}

// VPT: vectors of eight columns a thread keeps in registers; 0: rows too long
// for that are read again for each use.
template <class T, class W, bool EIGHT, int VPT>
__global__ void __launch_bounds__(1024) norm_kernel(NormKArgs a) {
  __shared__ double sums[16];
  __shared__ uint32_t tops[16];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
  const int H = a.hidden;
  const uint16_t* x = a.x + r * a.x_stride;
  const uint16_t* res = a.residual ? a.residual + r * a.residual_stride : nullptr;
  const W* weight = static_cast<const W*>(a.weight);

  auto total = [&](int c, int have, float (&s)[8]) {      // x + residual
    load_row8<T>(x + c, have, s);
    if (res) {
      float v[8];
      load_row8<T>(res + c, have, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
  };
  auto squares = [](const float (&s)[8]) {
    double q = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) q = __builtin_fma((double)s[e], (double)s[e], q);
    return q;
  };

  constexpr int kHeld = VPT > 0 ? VPT : 1;
  const int vectors = (H + 7) / 8;
  float s[kHeld][8];
  double q = 0;
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * threads + tid) * 8;
      if (c < H) total(c, H - c, s[i]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) s[i][e] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) q += squares(s[i]);
  } else {
    for (int c = tid * 8; c < H; c += threads * 8) {
      total(c, H - c, s[0]);
      q += squares(s[0]);
    }
  }
  const double rstd = 1.0 / sqrt(block_sum(q, sums, waves) / H + (double)a.eps);
  // For 16 bits a power of two of the factor goes apart where it is outside the
  // middle of float32's range.  For 8 bits it always does, and the rest stays
  // out of the values, whose quotients do not need it.
  const bool usual = rstd > 0 && rstd < 1e300, far = usual && (rstd < 0x1p-96 || rstd > 0x1p96);
  const int ex = (EIGHT ? usual : far) ? min(max(ilogb(rstd), -126), 126) : 0;
  const double rest = ldexp(rstd, -ex);
  const float r1 = EIGHT && !usual ? (float)rstd : ldexpf(1.0f, ex), r2 = (float)rest;

  auto scaled = [&](int c, int have, float (&v)[8]) {     // s to y; for 8 bits to y / rest
    float w[8];
    if constexpr (sizeof(W) == 4) load_row8(reinterpret_cast<const float*>(weight) + c, have, w);
    else load_row8<T>(reinterpret_cast<const uint16_t*>(weight) + c, have, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = EIGHT ? v[e] * r1 * w[e] : (far ? v[e] * r1 : v[e]) * r2 * w[e];
  };
  auto keep = [&](int c, int have, const float (&v)[8]) {
    if (a.residual_out) store_row8<T>(a.residual_out + r * a.residual_out_stride + c, have, v);
  };

  if constexpr (!EIGHT) {
    uint16_t* out = static_cast<uint16_t*>(a.out) + r * a.out_stride;
    if constexpr (VPT > 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * threads + tid) * 8;
        if (c < H) {
          keep(c, H - c, s[i]);
          scaled(c, H - c, s[i]);
          store_row8<T>(out + c, H - c, s[i]);
        }
      }
    } else {
      for (int c = tid * 8; c < H; c += threads * 8) {
        total(c, H - c, s[0]);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = s[0][e];
        scaled(c, H - c, y);
        keep(c, H - c, s[0]);
        store_row8<T>(out + c, H - c, y);
      }
    }
  } else {
    uint8_t* out = static_cast<uint8_t*>(a.out) + r * a.out_stride;
    float* scales = a.scales + r * a.scales_stride;
    auto top8 = [](const float (&y)[8]) {
      uint32_t t = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) t = max(t, magnitude(y[e]));
      return t;
    };
    const double share = usual ? rest / 448 : 1.0 / 448;
    const float m = usual ? r2 : 1.0f;
    auto scale_of = [&](uint32_t t) { return (float)(__uint_as_float(t) * share); };
    auto put = [&](int c, int have, float (&y)[8], uint32_t t) {
      divide(y, __uint_as_float(t), scale_of(t), m);
      store_e4m3(out + c, have, y);
    };
    // The lanes of a group of columns are neighbours: the maximum of theirs.
    const int lanes = a.group / 8;
    auto group_top = [&](uint32_t t, int c) {
      for (int d = 1; d < lanes; d *= 2) t = max(t, (uint32_t)__shfl_xor((int)t, d));
      if (c < H && c % a.group == 0) scales[c / a.group] = scale_of(t);
      return t;
    };
    if constexpr (VPT > 0) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * threads + tid) * 8;
        if (c < H) {
          keep(c, H - c, s[i]);
          scaled(c, H - c, s[i]);
        }
        uint32_t t = top8(s[i]);
        top = max(top, t);
        if (a.group) {
          t = group_top(t, c);
          if (c < H) put(c, H - c, s[i], t);
        }
      }
      if (!a.group) {
        top = block_max(top, tops, waves);
        if (tid == 0) scales[0] = scale_of(top);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = (i * threads + tid) * 8;
          if (c < H) put(c, H - c, s[i], top);
        }
      }
    } else {
      uint32_t top = 0;
      if (!a.group) {
        for (int c = tid * 8; c < H; c += threads * 8) {
          total(c, H - c, s[0]);
          scaled(c, H - c, s[0]);
          top = max(top, top8(s[0]));
        }
        top = block_max(top, tops, waves);
        if (tid == 0) scales[0] = scale_of(top);
      }
      for (int v = tid; v < (vectors + threads - 1) / threads * threads; v += threads) {   // all lanes take part
        const int c = v * 8;
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (c < H) {
          total(c, H - c, s[0]);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = s[0][e];
          scaled(c, H - c, y);
          keep(c, H - c, s[0]);
        }
        const uint32_t t = a.group ? group_top(top8(y), c) : top;
        if (c < H) put(c, H - c, y, t);
      }
    }
  }
}

template <class T, class W, bool EIGHT>
hipError_t launch(const NormKArgs& all, hipStream_t stream) {
  // Two vectors of a row to a thread where there are rows enough to hide each
  // other's latency (4096 rows of 7168 to 8 bits: 56 us with one, 47 with two,
  // 51 with four; 8192 of 4096 in 16 bits: 49, 51 and 54); one for few rows,
  // and four, or none held, where a workgroup has no more threads.
  const int vectors = (all.hidden + 7) / 8;
  int vpt = all.n >= 512 ? 2 : 1;
  while (vpt < 4 && vectors > 1024 * vpt) vpt *= 2;
  int threads = std::min((vectors + vpt - 1) / vpt, 1024);
  threads = (threads + 63) / 64 * 64;
  vpt = (vectors + threads - 1) / threads;
  // A launch has fewer than 2^32 threads.
  const int64_t most = ((int64_t)1 << 31) / threads;
  for (int64_t r = 0; r < all.n; r += most) {
    NormKArgs a = all;
    a.n = (int32_t)std::min<int64_t>(most, all.n - r);
    a.x += r * a.x_stride;
    if (a.residual) a.residual += r * a.residual_stride;
    a.out = static_cast<uint8_t*>(a.out) + r * a.out_stride * (EIGHT ? 1 : 2);
    if (a.scales) a.scales += r * a.scales_stride;
    if (a.residual_out) a.residual_out += r * a.residual_out_stride;
    const dim3 grid(a.n), block(threads);
    if (vpt <= 1) norm_kernel<T, W, EIGHT, 1><<<grid, block, 0, stream>>>(a);
    else if (vpt <= 2) norm_kernel<T, W, EIGHT, 2><<<grid, block, 0, stream>>>(a);
    else if (vpt <= 4) norm_kernel<T, W, EIGHT, 4><<<grid, block, 0, stream>>>(a);
    else norm_kernel<T, W, EIGHT, 0><<<grid, block, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class T>
hipError_t launch(const NormKArgs& a, bool weight_f32, bool eight, hipStream_t stream) {
  if (weight_f32) return eight ? launch<T, float, true>(a, stream) : launch<T, float, false>(a, stream);
  return eight ? launch<T, uint16_t, true>(a, stream) : launch<T, uint16_t, false>(a, stream);
}

}  // namespace

hipError_t launch_rms_norm(const NormKArgs& a, int dtype, bool weight_f32, bool eight, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? launch<BF16>(a, weight_f32, eight, stream) : launch<F16>(a, weight_f32, eight, stream);
}

}  // namespace moe_ep_detail
