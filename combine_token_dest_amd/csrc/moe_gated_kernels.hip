// gfx950 kernels of the gated product h = silu(x Wg^T) * (x Wu^T) and of its
// gradients.
//
// Forward: one matrix product whose tiles pair 32 gate columns with the same
// 32 up columns, so that a lane holds both and makes h in registers
// (moe_gemm_device.h); for a backward pass it also writes both as they are.
// Backward, from these: d = [dh u silu'(g), dh silu(g)] by a pass over the
// elements, then dx = d W and dW = d^T x as two products.  8192 rows of 7168 x
// 2048: 397 us forward (1.21 PFLOP/s), then 38 + 457 + 442.
//
// g and u are kept as float32: rounded to bfloat16 they would add as much to
// the gradients' error as their own rounding does (8192 rows of 7168 x 2048,
// off by 0.0030 of the norm where float32 leaves 0.0024), for 2% of the time.
// d goes into the products in the inputs' type, which the matrix instructions
// take.  Rounded once it adds half a step of an element to the same half step
// that dx and dW are rounded by (8192 rows of 7168 x 2048: off by 0.0023 of the
// norm, where a float32 d leaves 0.0017; float16 0.00029 and 0.00021).  With the
// rest of each rounding as a second part, whose products are added first, that
// part of the error is gone, for twice the products (forward and backward 1297 -> 2110 us).
// float16 would lose what is small and turn what is large into
// infinities, so there d is multiplied with a power of two that puts its
// largest element at 2^14 .. 2^15, and the products with its inverse.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "moe_dense_internal.h"
#include "moe_few_device.h"
#include "moe_gemm_device.h"

namespace moe_ep_detail {
namespace {

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + __expf(-v)); }

template <class G>
__global__ void __launch_bounds__(G::kThreads, G::kThreads / 256) gated_kernel(GatedKArgs a) {
  typedef typename G::T T;
  __shared__ __attribute__((aligned(1024))) char lds[G::kLds];
  int pt, qt;
  tile_of(a.ptiles, a.qtiles, &pt, &qt);
  typename G::SideP sp;
  typename G::SideQ sq;
  sp.aim(a.w, pt * (G::TP / 2));
  sq.aim(a.x, qt * G::TQ);
  G::begin((MOE_EP_LDS char*)lds, sp, sq, a.hidden);
  typename G::Acc acc;
  G::clear(acc);
  G::loop((MOE_EP_LDS char*)lds, sp, sq, a.hidden, acc);
  if (!G::join((MOE_EP_LDS char*)lds, acc)) return;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < G::FQ; ++j) {
    const int q = qt * G::TQ + G::wave_q() + j * 16 + (lane & 15);
    if (q >= a.x.rows) continue;
#pragma unroll
    for (int i = 0; i < G::FP; i += 2) {
      const int c = pt * (G::TP / 2) + (G::wave_p() + i * 16) / 2 + (lane >> 4) * 4;
      float g[4], u[4], h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = acc[i][j][e];
        u[e] = acc[i + 1][j][e];
        h[e] = g[e] * sigmoid(g[e]) * u[e];
      }
      store4<T>(a.out, q * a.out_stride + c, a.out_f32, a.inter - c, h);
      if (a.pre) {
        store4<T>(a.pre, (int64_t)q * 2 * a.inter + c, true, a.inter - c, g);
        store4<T>(a.pre, ((int64_t)q * 2 + 1) * a.inter + c, true, a.inter - c, u);
      }
    }
  }
}

// The same for up to 16 NT rows (moe_few_device.h): eight gate rows and the
// same eight up rows to a workgroup.
template <class T, int NT, int WAVES>
__global__ void __launch_bounds__(WAVES * 64) gated_few_kernel(GatedKArgs a) {
  typedef Few<T, 1, NT, WAVES> F;
  constexpr int kSums = WAVES * NT * 1024;
  __shared__ __attribute__((aligned(1024))) char lds[kSums > WAVES * F::kLds ? kSums : WAVES * F::kLds];
  f32x4 (*sums)[NT][16][4] = reinterpret_cast<f32x4 (*)[NT][16][4]>(lds);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15;
  const int c0 = blockIdx.x * 8;
  F few;
  const int steps = a.hidden / 64, left = a.hidden % 64;
  few.aim([&](int, int r) { return a.w.p + ((int64_t)min(c0 + (r & 7), a.inter - 1) + (r & 8 ? a.inter : 0)) * a.w.stride; },
          [&](int t, int r) { return a.x.p + (int64_t)min(t * 16 + r, a.x.rows - 1) * a.x.stride; }, 0, steps,
          blockIdx.x, lds + wave * F::kLds);
  few.prime(wave, WAVES);
  f32x4 acc[1][NT] = {};
  few.run(wave, WAVES, acc);
  if (left && steps % WAVES == wave) few.tail(left, acc);
  __syncthreads();                                        // the waves' pieces of lds become the sums
#pragma unroll
  for (int t = 0; t < NT; ++t) sums[wave][t][i][lane >> 4] = acc[0][t];
  __syncthreads();
  const float* sum = reinterpret_cast<const float*>(lds);
  for (int o = threadIdx.x; o < a.x.rows * 8; o += WAVES * 64) {
    const int r = o >> 3, c = o & 7;
    if (c0 + c >= a.inter) continue;
    float g = 0, u = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      g += sum[(w * NT * 16 + r) * 16 + c];
      u += sum[(w * NT * 16 + r) * 16 + 8 + c];
    }
    const float h = g * sigmoid(g) * u;
    const int64_t at = r * a.out_stride + c0 + c;
    if (a.out_f32) static_cast<float*>(a.out)[at] = h;
    else static_cast<uint16_t*>(a.out)[at] = T::from_float(h);
    if (a.pre) {
      a.pre[(int64_t)r * 2 * a.inter + c0 + c] = g;
      a.pre[((int64_t)r * 2 + 1) * a.inter + c0 + c] = u;
    }
  }
}

// PARTS: a workgroup of a few results' tiles takes one of a.parts parts of k
// (blockIdx.y, in whole tiles of k) and leaves float32 sums for sum_kernel.
// REST: q's second part is gone through first, with the same p.
template <class G, bool PARTS, bool REST>
__global__ void __launch_bounds__(G::kThreads, G::kThreads / 256) product_kernel(ProductKArgs a) {
  typedef typename G::T T;
  __shared__ __attribute__((aligned(1024))) char lds[G::kLds];
  int pt, qt;
  tile_of(a.ptiles, a.qtiles, &pt, &qt);
  typename G::SideP sp;
  typename G::SideQ sq;
  sp.aim(a.p, pt * G::TP);
  sq.aim(a.q, qt * G::TQ);
  int k = a.k;
  if constexpr (PARTS) {
    const int steps = (a.k + G::kK - 1) / G::kK;
    const int first = (int)((int64_t)steps * blockIdx.y / a.parts), last = (int)((int64_t)steps * (blockIdx.y + 1) / a.parts);
    sp.skip(first);
    sq.skip(first);
    k = min(a.k, last * G::kK) - first * G::kK;
  }
  typename G::Acc acc;
  if constexpr (REST) {
    G::clear(acc);
    sq.move(a.q_rest);
    auto back = [&](int count) {
      sp.skip(-count);
      sq.skip(-count);
      sq.move(-a.q_rest);
    };
    auto between = [&]() {
      if constexpr (std::is_same<T, F16>::value) {
#pragma unroll
        for (int i = 0; i < G::FP; ++i)
#pragma unroll
          for (int j = 0; j < G::FQ; ++j) acc[i][j] *= 1.0f / kRestUpF16;
      }
    };
    G::loop_twice((MOE_EP_LDS char*)lds, sp, sq, k, acc, back, between);
  } else {
    G::begin((MOE_EP_LDS char*)lds, sp, sq, k);
    G::clear(acc);
    G::loop((MOE_EP_LDS char*)lds, sp, sq, k, acc);
  }
  if (!G::join((MOE_EP_LDS char*)lds, acc)) return;
  const float factor = !PARTS && a.factor ? *a.factor : 1.0f;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < G::FQ; ++j) {
    const int q = qt * G::TQ + G::wave_q() + j * 16 + (lane & 15);
    if (q >= a.q_rows) continue;
#pragma unroll
    for (int i = 0; i < G::FP; ++i) {
      const int c = pt * G::TP + G::wave_p() + i * 16 + (lane >> 4) * 4;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * factor;
      if constexpr (PARTS)
        store4<T>(a.partial, ((int64_t)blockIdx.y * a.q_rows + q) * a.p.rows + c, true, a.p.rows - c, v);
      else
        store4<T>(a.out, q * a.out_stride + c, false, a.p.rows - c, v);
    }
  }
}

// out = *factor * the parts' sums, added in turn.
template <class T>
__global__ void __launch_bounds__(256) sum_kernel(ProductKArgs a) {
  const int64_t total = (int64_t)a.q_rows * a.p.rows;
  const float factor = a.factor ? *a.factor : 1.0f;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    float v = 0;
    for (int part = 0; part < a.parts; ++part) v += a.partial[part * total + i];
    const int64_t q = i / a.p.rows;
    a.out[q * a.out_stride + (i - q * a.p.rows)] = T::from_float(v * factor);
  }
}

// Elements c .. c + 7 (those below n) of a row of 16-bit or float32 numbers.
template <class T>
__device__ __forceinline__ void read8(const void* p, int64_t at, bool f32, int have, float (&v)[8]) {
  if (f32) {
    struct __attribute__((packed, aligned(4))) Four {
      f32x4 v;
    };
    const float* s = static_cast<const float*>(p) + at;
    if (have >= 8) {
      const f32x4 a = reinterpret_cast<const Four*>(s)->v, b = reinterpret_cast<const Four*>(s + 4)->v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[e + 4] = b[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < have ? s[e] : 0.0f;
    }
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(p) + at;
    if (have >= 8) {
      const u32x4 w = load_any8(s);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = T::to_float((uint16_t)w[e]);
        v[2 * e + 1] = T::to_float((uint16_t)(w[e] >> 16));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < have ? T::to_float(s[e]) : 0.0f;
    }
  }
}

template <class T>
__device__ __forceinline__ void write8(uint16_t* p, int have, const float (&v)[8]) {
  if (have >= 8) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = (uint32_t)T::from_float(v[2 * e]) | (uint32_t)T::from_float(v[2 * e + 1]) << 16;
    reinterpret_cast<AnyHalf8*>(p)->v = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < have) p[e] = T::from_float(v[e]);
  }
}

// What rounding to T leaves of each number (nothing of one that it makes
// infinite), in the scale that T keeps it in.
template <class T>
__device__ __forceinline__ void rests(float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float near = T::to_float(T::from_float(v[e])), rest = v[e] - near;
    v[e] = __builtin_isfinite(near) ? rest * (std::is_same<T, F16>::value ? kRestUpF16 : 1.0f) : 0.0f;
  }
}

// Eight columns of dgate and dup.
template <class T>
__device__ __forceinline__ void gate_grads(const GatedGradKArgs& a, int64_t row, int c, float (&dg)[8], float (&du)[8]) {
  const int have = a.inter - c;
  float dh[8], g[8], u[8];
  read8<T>(a.dout, row * a.dout_stride + c, a.dout_f32, have, dh);
  read8<T>(a.pre, row * 2 * a.inter + c, true, have, g);
  read8<T>(a.pre, (row * 2 + 1) * a.inter + c, true, have, u);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float s = sigmoid(g[e]);
    dg[e] = e < have ? dh[e] * u[e] * (s * (1.0f + g[e] * (1.0f - s))) : 0.0f;
    du[e] = e < have ? dh[e] * (g[e] * s) : 0.0f;
  }
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

// The largest finite magnitude in d that each workgroup meets.
template <class T>
__global__ void __launch_bounds__(256) gated_top_kernel(GatedGradKArgs a) {
  __shared__ uint32_t part[4];
  const int vectors = (a.inter + 7) / 8;
  const int64_t total = (int64_t)a.n * vectors;
  uint32_t top = 0;
  for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < total; v += (int64_t)gridDim.x * 256) {
    const int64_t row = v / vectors;
    float dg[8], du[8];
    gate_grads<T>(a, row, (int)(v - row * vectors) * 8, dg, du);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = __float_as_uint(dg[e]) & 0x7FFFFFFFu, y = __float_as_uint(du[e]) & 0x7FFFFFFFu;
      top = max(top, max(x < 0x7F800000u ? x : 0u, y < 0x7F800000u ? y : 0u));
    }
  }
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) a.tops[blockIdx.x] = max(max(part[0], part[1]), max(part[2], part[3]));
}

// `tops` partial maxima (float16), then d.
template <class T>
__global__ void __launch_bounds__(256) gated_grad_kernel(GatedGradKArgs a, int tops) {
  float up = 1.0f;
  if constexpr (std::is_same<T, F16>::value) {
    __shared__ uint32_t part[4];
    uint32_t top = 0;
    for (int i = threadIdx.x; i < tops; i += 256) top = max(top, a.tops[i]);
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    const int ex = top ? min(max(14 - ilogbf(__uint_as_float(top)), -126), 126) : 0;
    up = ldexpf(1.0f, ex);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.factor = ldexpf(1.0f, -ex);
  }
  const int vectors = (a.inter + 7) / 8;
  const int64_t total = (int64_t)a.n * vectors;
  for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < total; v += (int64_t)gridDim.x * 256) {
    const int64_t row = v / vectors;
    const int c = (int)(v - row * vectors) * 8;
    float dg[8], du[8];
    gate_grads<T>(a, row, c, dg, du);
    if constexpr (std::is_same<T, F16>::value) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dg[e] *= up;
        du[e] *= up;
      }
    }
    uint16_t* d = a.d + row * a.d_stride + c;
    write8<T>(d, a.inter - c, dg);
    write8<T>(d + a.inter, a.inter - c, du);
    if (a.rest) {
      uint16_t* r = a.rest + row * a.d_stride + c;
      rests<T>(dg);
      rests<T>(du);
      write8<T>(r, a.inter - c, dg);
      write8<T>(r + a.inter, a.inter - c, du);
    }
  }
}

template <class G>
hipError_t gated_tiles(GatedKArgs a, hipStream_t stream) {
  a.ptiles = tiles(a.inter, G::TP / 2);
  a.qtiles = tiles(a.x.rows, G::TQ);
  gated_kernel<G><<<dim3(a.ptiles * a.qtiles), dim3(G::kThreads), 0, stream>>>(a);
  return hipGetLastError();
}
template <class T, int NT>
hipError_t gated_few(const GatedKArgs& a, hipStream_t stream) {
  const int blocks = tiles(a.inter, 8);
  if (NT > 2 || blocks >= 256) gated_few_kernel<T, NT, 8><<<dim3(blocks), dim3(512), 0, stream>>>(a);
  else gated_few_kernel<T, NT <= 2 ? NT : 2, 16><<<dim3(blocks), dim3(1024), 0, stream>>>(a);
  return hipGetLastError();
}
template <class T>
hipError_t gated(const GatedKArgs& a, hipStream_t stream) {
  if (a.x.rows <= 16) return gated_few<T, 1>(a, stream);
  if (a.x.rows <= 32) return gated_few<T, 2>(a, stream);
  if (a.x.rows <= gated_few_rows(a.inter))
    return a.x.rows <= 48 ? gated_few<T, 3>(a, stream) : gated_few<T, 4>(a, stream);
  const bool direct = a.w.whole && a.x.whole;
  switch (tile_size(2 * (int64_t)a.inter, a.x.rows, a.hidden, direct, true)) {
    case k256x256: return gated_tiles<Gemm<T, true, true, true, 256, 256, 2, 4, 1, true>>(a, stream);
    case k256x128: return gated_tiles<Gemm<T, true, true, true, 256, 128, 2, 4, 1, true>>(a, stream);
    case k128x128:
      return direct ? gated_tiles<Gemm<T, true, true, true, 128, 128, 2, 2, 2, true>>(a, stream)
                    : gated_tiles<Gemm<T, true, true, true, 128, 128, 2, 2, 2, false>>(a, stream);
    case k64x64:
      return direct ? gated_tiles<Gemm<T, true, true, true, 64, 64, 2, 2, 4, true>>(a, stream)
                    : gated_tiles<Gemm<T, true, true, true, 64, 64, 2, 2, 4, false>>(a, stream);
    default:
      return direct ? gated_tiles<Gemm<T, true, true, true, 32, 32, 1, 1, 4, true>>(a, stream)
                    : gated_tiles<Gemm<T, true, true, true, 32, 32, 1, 1, 4, false>>(a, stream);
  }
}

template <class G>
hipError_t product_tiles(ProductKArgs a, hipStream_t stream) {
  a.ptiles = tiles(a.p.rows, G::TP);
  a.qtiles = tiles(a.q_rows, G::TQ);
  const int count = a.ptiles * a.qtiles;
  if constexpr (G::TP == 64) {
    static_assert(G::TQ == 64 && G::kK == 256, "product_parts()");
    const int64_t results = (int64_t)a.p.rows * a.q_rows;
    a.parts = product_parts(a.p.rows, a.q_rows, a.k);
    if (a.parts > 1) {
      const dim3 grid(count, a.parts), block(G::kThreads);
      if (a.q_rest) product_kernel<G, true, true><<<grid, block, 0, stream>>>(a);
      else product_kernel<G, true, false><<<grid, block, 0, stream>>>(a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      sum_kernel<typename G::T><<<dim3((int)std::min<int64_t>((results + 255) / 256, 2048)), dim3(256), 0, stream>>>(a);
      return hipGetLastError();
    }
  }
  if (a.q_rest) product_kernel<G, false, true><<<dim3(count), dim3(G::kThreads), 0, stream>>>(a);
  else product_kernel<G, false, false><<<dim3(count), dim3(G::kThreads), 0, stream>>>(a);
  return hipGetLastError();
}
template <class T, bool QKC>
hipError_t product(const ProductKArgs& a, hipStream_t stream) {
  const bool direct = a.p.whole && a.q.whole;
  switch (tile_size(a.p.rows, a.q_rows, a.q_rest ? 2 * (int64_t)a.k : a.k, direct, false)) {
    case k256x256: return product_tiles<Gemm<T, false, QKC, false, 256, 256, 2, 4, 1, true>>(a, stream);
    case k256x128: return product_tiles<Gemm<T, false, QKC, false, 256, 128, 2, 4, 1, true>>(a, stream);
    case k128x128:
      return direct ? product_tiles<Gemm<T, false, QKC, false, 128, 128, 2, 2, 2, true>>(a, stream)
                    : product_tiles<Gemm<T, false, QKC, false, 128, 128, 2, 2, 2, false>>(a, stream);
    default:
      return direct ? product_tiles<Gemm<T, false, QKC, false, 64, 64, 2, 2, 4, true>>(a, stream)
                    : product_tiles<Gemm<T, false, QKC, false, 64, 64, 2, 2, 4, false>>(a, stream);
  }
}

template <class T>
hipError_t gated_grad(const GatedGradKArgs& a, hipStream_t stream) {
  const int64_t vectors = (int64_t)a.n * ((a.inter + 7) / 8);
  const int blocks = (int)std::min<int64_t>((vectors + 255) / 256, 8192);
  const int tops = std::min(blocks, kTops);
  if (std::is_same<T, F16>::value) {
    gated_top_kernel<T><<<dim3(tops), dim3(256), 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  gated_grad_kernel<T><<<dim3(blocks), dim3(256), 0, stream>>>(a, tops);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated(const GatedKArgs& a, int dtype, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? gated<BF16>(a, stream) : gated<F16>(a, stream);
}

hipError_t launch_gated_grad(const GatedGradKArgs& a, int dtype, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? gated_grad<BF16>(a, stream) : gated_grad<F16>(a, stream);
}

hipError_t launch_product(const ProductKArgs& a, int dtype, bool q_kc, hipStream_t stream) {
  if (dtype == MOE_EP_BF16) return q_kc ? product<BF16, true>(a, stream) : product<BF16, false>(a, stream);
  return q_kc ? product<F16, true>(a, stream) : product<F16, false>(a, stream);
}

}  // namespace moe_ep_detail
