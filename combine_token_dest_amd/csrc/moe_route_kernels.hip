// gfx950 kernel of the router's selection (moe_ep_route).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <climits>
#include <type_traits>

#include "moe_experts_device.h"
#include "moe_experts_internal.h"

namespace moe_ep_detail {
namespace {

__device__ __forceinline__ float load_logit(const void* p, int64_t i, int dtype) {
  if (dtype == MOE_EP_F32) return static_cast<const float*>(p)[i];
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  return dtype == MOE_EP_BF16 ? BF16::to_float(v) : F16::to_float(v);
}

// -inf closes the expert; NaN does too; +inf reads as the largest float.
__device__ __forceinline__ float clean_logit(float l) {
  return l == l ? __builtin_fminf(l, FLT_MAX) : -INFINITY;
}

template <typename V>
__device__ __forceinline__ bool better(V v1, int e1, V v0, int e0) {
  return v1 > v0 || (v1 == v0 && e1 < e0);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(x)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
  u32x2 u = __builtin_bit_cast(u32x2, x);
  u[0] = dpp<CTRL>(u[0]);
  u[1] = dpp<CTRL>(u[1]);
  return __builtin_bit_cast(double, u);
}

// x of both halves of a pair of 16-lane rows (W = 16) or of a pair of 32-lane
// halves (W = 32): the two results are the pair's first and second member.
template <int W>
__device__ __forceinline__ void both(uint32_t x, uint32_t* a, uint32_t* b) {
  if constexpr (W == 16) {
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    *a = r[0];
    *b = r[1];
  } else {
    auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    *a = r[0];
    *b = r[1];
  }
}
template <int W>
__device__ __forceinline__ void both(float x, float* a, float* b) {
  uint32_t u, v;
  both<W>(__float_as_uint(x), &u, &v);
  *a = __uint_as_float(u);
  *b = __uint_as_float(v);
}
template <int W>
__device__ __forceinline__ void both(double x, double* a, double* b) {
  const u32x2 u = __builtin_bit_cast(u32x2, x);
  u32x2 p, q;
  uint32_t s, t;
  both<W>(u[0], &s, &t);
  p[0] = s;
  q[0] = t;
  both<W>(u[1], &s, &t);
  p[1] = s;
  q[1] = t;
  *a = __builtin_bit_cast(double, p);
  *b = __builtin_bit_cast(double, q);
}

// All-reductions over the LPT (16 or 64) lanes of a token.
template <int CTRL, typename V>
__device__ __forceinline__ void best_step(V& v, int& e) {
  const V ov = dpp<CTRL>(v);
  const int oe = (int)dpp<CTRL>((uint32_t)e);
  if (better(ov, oe, v, e)) {
    v = ov;
    e = oe;
  }
}
template <int W, typename V>
__device__ __forceinline__ void best_pair(V& v, int& e) {
  V a, b;
  uint32_t ea, eb;
  both<W>(v, &a, &b);
  both<W>((uint32_t)e, &ea, &eb);
  const bool second = better(b, (int)eb, a, (int)ea);
  v = second ? b : a;
  e = second ? (int)eb : (int)ea;
}
template <int LPT, typename V>
__device__ __forceinline__ void reduce_best(V& v, int& e) {
  best_step<0x128>(v, e);   // row_ror:8, 4, 2, 1
  best_step<0x124>(v, e);
  best_step<0x122>(v, e);
  best_step<0x121>(v, e);
  if constexpr (LPT == 64) {
    best_pair<16>(v, e);
    best_pair<32>(v, e);
  }
}
template <int LPT, typename V>
__device__ __forceinline__ V reduce_sum(V v) {
  v += dpp<0x128>(v);
  v += dpp<0x124>(v);
  v += dpp<0x122>(v);
  v += dpp<0x121>(v);
  if constexpr (LPT == 64) {
    V a, b;
    both<16>(v, &a, &b);
    v = a + b;
    both<32>(v, &a, &b);
    v = a + b;
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float reduce_max(float v) {
  int e = 0;
  reduce_best<LPT>(v, e);
  return v;
}

__device__ __forceinline__ double score64(int score, float l, float top) {
  return score == MOE_EP_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top);
}

constexpr int kRouteThreads = 256;

// One token per LPT lanes, expert e = v * LPT + lane in register v.  The
// selection is top_k rounds of an all-lane maximum of (choice, lowest index).
// Without a bias or groups the choice is the logit itself (V = float): it
// orders the experts as the score does, without the ties of a saturated
// score.  Otherwise it is the score in float64 (V = double), so that a
// near-tie is decided by the values and not by a float32 rounding.
// Weights are computed in float64 by one lane per slot and rounded once.
template <typename V, int LPT, int VPL, bool GROUPS>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteKArgs a) {
  constexpr int kTokens = 64 / LPT;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int sub = lane & (LPT - 1);
  const int64_t token = ((int64_t)blockIdx.x * (kRouteThreads / 64) + wave) * kTokens + lane / LPT;
  const int64_t t = token < a.n ? token : a.n - 1;
  const int E = a.num_experts;
  const int64_t row = t * a.logits_stride;

  float l[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = v * LPT + sub;
    l[v] = load_logit(a.logits, row + (e < E ? e : E - 1), a.logits_dtype);
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) l[v] = v * LPT + sub < E ? clean_logit(l[v]) : -INFINITY;

  V c[VPL];
  float top = 0.0f;
  double total = 1.0;
  if constexpr (std::is_same<V, double>::value) {
    if (a.score == MOE_EP_SCORE_SOFTMAX) {
      float m = l[0];
#pragma unroll
      for (int v = 1; v < VPL; ++v) m = __builtin_fmaxf(m, l[v]);
      top = reduce_max<LPT>(m);
      double s = 0.0;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        c[v] = l[v] == -INFINITY ? 0.0 : score64(MOE_EP_SCORE_SOFTMAX, l[v], top);
        s += c[v];
      }
      total = reduce_sum<LPT>(s);
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = v * LPT + sub;
      double x = a.score == MOE_EP_SCORE_SOFTMAX ? c[v] / total : score64(MOE_EP_SCORE_SIGMOID, l[v], 0.0f);
      if (a.bias) x += (double)a.bias[e < E ? e : E - 1];
      c[v] = l[v] > -INFINITY && x > -INFINITY ? x : -INFINITY;   // a NaN bias closes too
    }
    if constexpr (GROUPS) {
      // LPT is 64 here: one token per wave.
      extern __shared__ double lds[];
      const int G = a.num_groups;
      const int size = E / G;
      double* cs = lds + wave * (E + G);
      double* gv = cs + E;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int e = v * LPT + sub;
        if (e < E) cs[e] = c[v];
      }
      __syncthreads();
      for (int g = sub; g < G; g += LPT) {
        double b1 = -INFINITY, b2 = -INFINITY;
        for (int i = 0; i < size; ++i) {
          const double x = cs[g * size + i];
          if (x > b1) {
            b2 = b1;
            b1 = x;
          } else if (x > b2) {
            b2 = x;
          }
        }
        gv[g] = a.group_top > 1 && b2 > -INFINITY ? b1 + b2 : b1;
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int e = v * LPT + sub;
        if (e < E) {
          const int g = e / size;
          const double mine = gv[g];
          int ahead = 0;
          for (int h = 0; h < G; ++h) ahead += better(gv[h], h, mine, g) ? 1 : 0;
          if (ahead >= a.top_groups) c[v] = -INFINITY;
        }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) c[v] = l[v];
  }

  int mine = INT_MAX;       // the expert of slot `sub`
  for (int r = 0; r < a.top_k; ++r) {
    V bv = -INFINITY;
    int be = INT_MAX;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (c[v] > bv) {
        bv = c[v];
        be = v * LPT + sub;
      }
    }
    reduce_best<LPT>(bv, be);
    if (std::is_same<V, float>::value && r == 0) top = (float)bv;
    if (sub == r) mine = be;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (be == v * LPT + sub) c[v] = -INFINITY;
    }
  }

  if constexpr (std::is_same<V, float>::value) {
    if (a.score == MOE_EP_SCORE_SOFTMAX && !a.renormalize) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) s += l[v] == -INFINITY ? 0.0f : expf(l[v] - top);
      total = (double)reduce_sum<LPT>(s);
    }
  }
  const bool open = mine != INT_MAX && sub < a.top_k;
  double s = 0.0;
  if (open) s = score64(a.score, clean_logit(load_logit(a.logits, row + mine, a.logits_dtype)), top);
  const double z = a.renormalize ? reduce_sum<LPT>(s) : total;
  if (token < a.n && sub < a.top_k) {
    a.ids[token * a.top_k + sub] = open ? mine : a.invalid_id;
    a.weights[token * a.top_k + sub] = z > 0.0 ? (float)(s / z * (double)a.scale) : 0.0f;
  }
}

template <typename V, int LPT, bool GROUPS>
void start_route(const RouteKArgs& a, hipStream_t stream) {
  constexpr int kPerBlock = kRouteThreads / 64 * (64 / LPT);
  const int grid = (int)(((int64_t)a.n + kPerBlock - 1) / kPerBlock);
  const size_t lds = GROUPS ? (size_t)(kRouteThreads / 64) * (a.num_experts + a.num_groups) * sizeof(double) : 0;
  const int vpl = (a.num_experts + LPT - 1) / LPT;
  if (vpl <= 1) route_kernel<V, LPT, 1, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
  else if (vpl <= 2) route_kernel<V, LPT, 2, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
  else if (vpl <= 4) route_kernel<V, LPT, 4, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
  else if (vpl <= 8) route_kernel<V, LPT, 8, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
  else route_kernel<V, LPT, 16, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
}

}  // namespace

hipError_t launch_route(const RouteKArgs& a, hipStream_t stream) {
  if (a.num_groups > 1) start_route<double, 64, true>(a, stream);
  else if (a.bias) start_route<double, 64, false>(a, stream);
  else start_route<float, 64, false>(a, stream);
  return hipGetLastError();
}

}  // namespace moe_ep_detail
