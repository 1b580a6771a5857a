// gfx950 kernel of the root-mean-square norm with the residual's addition:
// s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, the rows leaving
// in 16 bits or as e4m3 with a scale for each group of columns.
//
// One read of x and residual and one write of each output is all it has to
// move (8-bit rows with a residual: 7 bytes a column), so it is bound by memory:
// the kernel for 8192 rows of 4096 in 16 bits takes 46 us (5.8 TB/s; a copy of
// 2 GiB, half of it writes, runs at 4.9) and for 4096 of 7168 with a residual to
// 8 bits 46 (4.5).  A workgroup takes one row and keeps s in registers between
// the sum of squares and the outputs; the squares are summed in float64, which
// hides behind the loads and cannot overflow.
//
// Maxima of magnitudes are taken over the bits as integers: NaN is above
// infinity there, so it is not lost, as it would be in a float maximum.
//
// The 8-bit values are the nearest ones to 448 s w / max|s w|.  float32 tells for
// all but one in 2^16 (with 16-bit weights, whose quotients often lie in a
// middle itself, one in 2^13); those are settled by float64 products, which are
// whole.  A value on the wrong side of a middle is off by a sixteenth of itself, and
// some few of a million were (of 8 million with float32 weights 21): 1 to 2 us
// of the 44 above with a scale a group, and of 42 with a scale a row.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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

// Eight values as e4m3, to nearest even; NaN stays NaN.
__device__ __forceinline__ u32x2 e4m3(const float (&q)[8]) {
  u32x2 w = {0, 0};
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    w[e >> 1] = __builtin_amdgcn_cvt_pk_fp8_f32(q[2 * e], q[2 * e + 1], w[e >> 1], false);
    w[e >> 1] = __builtin_amdgcn_cvt_pk_fp8_f32(q[2 * e + 2], q[2 * e + 3], w[e >> 1], true);
  }
  return w;
}
__device__ __forceinline__ void store_e4m3(uint8_t* p, int have, const u32x2& w) {
  if (have >= 8) {
    reinterpret_cast<Byte8*>(p)->v = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < have) p[e] = (uint8_t)(w[e >> 2] >> (e & 3) * 8);
  }
}

// 448 v / top as e4m3, of a group with the largest magnitude top, whose scale is
// m top / 448.  Each v and top is off by one rounding; with those of the
// quotient that is at most 5 x 2^-24 of it, so where 2^-21 more and less round to
// the same value, that is the quotient's, whatever the roundings were.
// Elsewhere the two differ, for settle().  A scale near
// float32's end may be rounded by any share, so there it is what is divided by,
// brought up by 2^100 as v is, and the quotient needs an end.
__device__ __forceinline__ void quotients(const float (&v)[8], float top, float scale, float m, u32x2* more, u32x2* less) {
  float a[8];
  if (scale < 0x1p-64f) {
    const float inv = scale == 0.0f ? 0.0f : m / (scale * 0x1p100f);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = fminf(fmaxf(v[e] * 0x1p100f * inv, -448.0f), 448.0f);
    *more = *less = e4m3(a);
    return;
  }
  const float factor = 448.0f / top;                       // 0 of an infinity, NaN of NaN
  const float high = factor * (1.0f + 0x1p-21f), low = factor * (1.0f - 0x1p-21f);
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = v[e] * high;
  *more = e4m3(a);
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = v[e] * low;
  *less = e4m3(a);
}

// Which of two neighbouring e4m3 values is 448 |s w| / top's, where they differ:
// the products on both sides of the middle between them, 896 |s w| and the
// values' sum times top, are whole in float64 (51 and 53 bits).  rounded: top may
// be off by a rounding to float32; false if that could matter.
__device__ __forceinline__ bool settle(const float (&s)[8], const float (&w)[8], double top, bool rounded,
                                       const u32x2& more, const u32x2& less, u32x2* out) {
  bool sure = true;
  const uint64_t high = (uint64_t)more[1] << 32 | more[0], low = (uint64_t)less[1] << 32 | less[0];
  uint64_t open = high ^ low, r = high;
  while (open) {
    const int at = __builtin_ctzll(open) & ~7;
    float se = s[0], we = w[0];
#pragma unroll
    for (int e = 1; e < 8; ++e)
      if (at == e * 8) {
        se = s[e];
        we = w[e];
      }
    const int h = (int)(high >> at) & 0x7F, l = (int)(low >> at) & 0x7F;
    const float sum = __builtin_amdgcn_cvt_f32_fp8(h, 0) + __builtin_amdgcn_cvt_f32_fp8(l, 0);
    const double whole = 896.0 * fabs((double)se * (double)we), middle = (double)sum * top;
    const uint64_t byte = (uint64_t)0xFF << at;
    if (whole < middle || (whole == middle && (h & 1))) r = (r & ~byte) | (low & byte);
    if (rounded && fabs(whole - middle) <= middle * 0x1.001p-24) sure = false;
    open &= ~byte;
  }
  *out = u32x2{(uint32_t)r, (uint32_t)(r >> 32)};
  return sure;
}

// Whether products with 16-bit weights are whole in float32 for sure: the
// factors have 24 significant bits together at most.  (They mostly are, and
// quotients in the very middle are common then.)
template <class T>
__device__ __forceinline__ bool all_whole(const float (&s)[8]) {
  constexpr uint32_t kBits = std::is_same<T, F16>::value ? 11 : 8;    // a weight's
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) bits |= __float_as_uint(s[e]);
  return !(bits & ((1u << kBits) - 1));
}

// What rounding left of the largest products: of those |s w| that are rounded
// to top, the most that is lacking (with the sign of its own).
__device__ __forceinline__ float rest_of_top(const float (&s)[8], const float (&w)[8], const float (&v)[8], float top) {
  float rest = -INFINITY;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (fabsf(v[e]) == top) rest = fmaxf(rest, __builtin_fmaf(fabsf(s[e]), fabsf(w[e]), -top));
  return rest;
}
// A float as a number above 0 that is larger for a larger one.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) { return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

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

enum Rows { kSixteen, kGroups, kWhole };                  // in 16 bits; in 8 with a scale a group, or a row

// VPT: vectors of eight columns a thread keeps in registers; 0: rows too long
// for that are read again for each use.  (Up to two leave room for two of the
// largest workgroups on a CU.)
template <class T, class W, Rows ROWS, int VPT>
__global__ void __launch_bounds__(1024, VPT <= 2 ? 8 : 4) norm_kernel(NormKArgs a) {
  constexpr bool EIGHT = ROWS != kSixteen;
  __shared__ double sums[16];
  __shared__ uint32_t tops[16];
  __shared__ uint32_t top_rest, any_open;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
  const int H = a.hidden;
  if (ROWS == kWhole && tid == 0) top_rest = any_open = 0;
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

  auto factors = [&](int c, int have, float (&w)[8]) {     // the weight
    if constexpr (sizeof(W) == 4) load_row8(reinterpret_cast<const float*>(weight) + c, have, w);
    else load_row8<T>(reinterpret_cast<const uint16_t*>(weight) + c, have, w);
  };
  auto keep = [&](int c, int have, const float (&v)[8]) {
    if (a.residual_out) store_row8<T>(a.residual_out + r * a.residual_out_stride + c, have, v);
  };

  if constexpr (!EIGHT) {
    auto scaled = [&](int c, int have, float (&v)[8]) {   // s to y
      float w[8];
      factors(c, have, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (far ? v[e] * r1 : v[e]) * r2 * w[e];
    };
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
    auto total_or_zero = [&](int c, float (&u)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = 0.0f;
      if (c < H) total(c, H - c, u);
    };
    // s with its power of two.
    auto scale = [&](float (&u)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] *= r1;
    };
    auto keep_and_scale = [&](int c, float (&u)[8]) {
      if (c < H) keep(c, H - c, u);
      scale(u);
    };
    // The weights and v = y / rest of a vector.  Past the row's end s is 0, and so
    // are they; where r1 is no number there, none of the row is.
    auto products = [&](int c, const float (&u)[8], float (&w)[8], float (&v)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 0.0f;
      if (c < H) factors(c, H - c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = u[e] * w[e];
    };
    // Writes a vector's values; whether some of the wave's are open.
    auto put = [&](int c, const float (&v)[8], uint32_t t, u32x2* more, u32x2* less) {
      quotients(v, __uint_as_float(t), scale_of(t), m, more, less);
      const bool open = __ballot((*more)[0] != (*less)[0] || (*more)[1] != (*less)[1]);
      if (c < H) store_e4m3(out + c, H - c, *more);
      return open;
    };
    // The open ones, with what the largest product lacks.
    auto put_open = [&](int c, const float (&u)[8], const float (&w)[8], uint32_t t, float lacking, const u32x2& more,
                        const u32x2& less) {
      u32x2 q;
      settle(u, w, (double)__uint_as_float(t) + (double)lacking, false, more, less, &q);
      if (c < H) store_e4m3(out + c, H - c, q);
    };
    // The lanes of a group of columns are neighbours: the maximum of theirs.
    const int lanes = a.group / 8;
    auto put_group = [&](int c, float (&u)[8]) {
      keep_and_scale(c, u);
      float w[8], v[8];
      products(c, u, w, v);
      uint32_t t = top8(v);
      for (int d = 1; d < lanes; d *= 2) t = max(t, (uint32_t)__shfl_xor((int)t, d));
      if (c < H && c % a.group == 0) scales[c / a.group] = scale_of(t);
      u32x2 more, less;
      if (put(c, v, t, &more, &less)) {
        float lacking = rest_of_top(u, w, v, __uint_as_float(t));
        for (int d = 1; d < lanes; d *= 2) lacking = fmaxf(lacking, __shfl_xor(lacking, d));
        put_open(c, u, w, t, lacking, more, less);
      }
    };
    if constexpr (ROWS == kGroups) {
      if constexpr (VPT > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) put_group((i * threads + tid) * 8, s[i]);
      } else {
        for (int v = tid; v < (vectors + threads - 1) / threads * threads; v += threads) {
          const int c = v * 8;
          total_or_zero(c, s[0]);
          put_group(c, s[0]);
        }
      }
    } else {
      uint32_t mine = 0;
      // The products stay in registers too, or are made again.
      constexpr bool kKeep = VPT == 1 || VPT == 2;
      float kept[kKeep ? VPT : 1][8];
      // A magnitude's 31 bits, and whether it may be rounded.
      auto find = [&](int c, const float (&u)[8], float (&v)[8]) {
        float w[8];
        products(c, u, w, v);
        mine = max(mine, top8(v) << 1 | (sizeof(W) == 2 && all_whole<T>(u) ? 0u : 1u));
      };
      if constexpr (VPT > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          keep_and_scale((i * threads + tid) * 8, s[i]);
          find((i * threads + tid) * 8, s[i], kept[kKeep ? i : 0]);
        }
      } else {
        for (int c = tid * 8; c < H; c += threads * 8) {
          total(c, H - c, s[0]);
          scale(s[0]);
          find(c, s[0], kept[0]);
        }
      }
      const uint32_t top_and_rounded = block_max(mine, tops, waves), t = top_and_rounded >> 1;
      const bool rounded = top_and_rounded & 1;
      if (tid == 0) scales[0] = scale_of(t);
      // What the largest products lack: the few threads that have one say it.
      auto lacking = [&](int c, const float (&u)[8]) {
        float w[8], v[8];
        products(c, u, w, v);
        atomicMax(&top_rest, ordered(rest_of_top(u, w, v, __uint_as_float(t))));
      };
      auto put_whole = [&](int c, const float (&u)[8], float (&v)[8]) {
        float w[8];
        if constexpr (!kKeep) products(c, u, w, v);
        u32x2 more, less, q;
        if (!put(c, v, t, &more, &less)) return false;
        float again[8];
        products(c, u, w, again);
        const bool sure = settle(u, w, (double)__uint_as_float(t), rounded, more, less, &q);
        if (c < H) store_e4m3(out + c, H - c, q);
        return __ballot(!sure) != 0;
      };
      auto put_whole_open = [&](int c, const float (&u)[8]) {
        float w[8], v[8];
        products(c, u, w, v);
        u32x2 more, less;
        if (put(c, v, t, &more, &less)) put_open(c, u, w, t, from_ordered(top_rest), more, less);
      };
      if constexpr (VPT > 0) {
        // Where the largest is rounded, that matters in one row of a hundred (4096
        // columns).
        bool open = false;
#pragma unroll
        for (int i = 0; i < VPT; ++i) open |= put_whole((i * threads + tid) * 8, s[i], kept[kKeep ? i : 0]);
        if (open) any_open = 1;
        __syncthreads();
        if (any_open) {
          if (mine >> 1 == t)
#pragma unroll
            for (int i = 0; i < VPT; ++i) lacking((i * threads + tid) * 8, s[i]);
          __syncthreads();
          if (open)
#pragma unroll
            for (int i = 0; i < VPT; ++i) put_whole_open((i * threads + tid) * 8, s[i]);
        }
      } else {
        // (The residual may be where x or the old one is: what reads them comes
        // before the first write.)
        if (mine >> 1 == t)
          for (int c = tid * 8; c < H; c += threads * 8) {
            total(c, H - c, s[0]);
            scale(s[0]);
            lacking(c, s[0]);
          }
        __syncthreads();
        for (int v = tid; v < (vectors + threads - 1) / threads * threads; v += threads) {
          const int c = v * 8;
          total_or_zero(c, s[0]);
          keep_and_scale(c, s[0]);
          put_whole_open(c, s[0]);
        }
      }
    }
  }
}

template <class T, class W, Rows ROWS>
hipError_t launch(const NormKArgs& all, hipStream_t stream) {
  // Two vectors of a row to a thread where there are rows enough to hide each
  // other's latency (calls of 4096 rows of 7168 to 8 bits: 56 us with one, 47 with
  // two, 51 with four; 8192 of 4096 in 16 bits: 49, 51 and 54); one for few rows,
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
    a.out = static_cast<uint8_t*>(a.out) + r * a.out_stride * (ROWS == kSixteen ? 2 : 1);
    if (a.scales) a.scales += r * a.scales_stride;
    if (a.residual_out) a.residual_out += r * a.residual_out_stride;
    const dim3 grid(a.n), block(threads);
    if (vpt <= 1) norm_kernel<T, W, ROWS, 1><<<grid, block, 0, stream>>>(a);
    else if (vpt <= 2) norm_kernel<T, W, ROWS, 2><<<grid, block, 0, stream>>>(a);
    else if (vpt <= 4) norm_kernel<T, W, ROWS, 4><<<grid, block, 0, stream>>>(a);
    else norm_kernel<T, W, ROWS, 0><<<grid, block, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class T, class W>
hipError_t launch(const NormKArgs& a, bool eight, hipStream_t stream) {
  if (!eight) return launch<T, W, kSixteen>(a, stream);
  return a.group ? launch<T, W, kGroups>(a, stream) : launch<T, W, kWhole>(a, stream);
}
template <class T>
hipError_t launch(const NormKArgs& a, bool weight_f32, bool eight, hipStream_t stream) {
  return weight_f32 ? launch<T, float>(a, eight, stream) : launch<T, uint16_t>(a, eight, stream);
}

}  // namespace

hipError_t launch_rms_norm(const NormKArgs& a, int dtype, bool weight_f32, bool eight, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? launch<BF16>(a, weight_f32, eight, stream) : launch<F16>(a, weight_f32, eight, stream);
}

}  // namespace moe_ep_detail
