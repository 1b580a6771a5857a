// The router's selection for one token, on the device: used by moe_ep_route's
// kernel and by the layer's first kernel for a few tokens.
#pragma once

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

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return __builtin_amdgcn_mov_dpp(x, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return (int)dpp<CTRL>((uint32_t)x);
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

// x of both members of a pair of 16-lane rows (W = 16) or of the pair of
// 32-lane halves (W = 32), in every lane of the pair.
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
__device__ __forceinline__ void both(int x, int* a, int* b) {
  uint32_t u, v;
  both<W>((uint32_t)x, &u, &v);
  *a = (int)u;
  *b = (int)v;
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

// All-reduction over the LPT (16 or 64) lanes of a token, in a fixed order.
template <int LPT, typename V, typename F>
__device__ __forceinline__ V reduce(V v, F op) {
  v = op(v, dpp<0x128>(v));             // row_ror:8, 4, 2, 1
  v = op(v, dpp<0x124>(v));
  v = op(v, dpp<0x122>(v));
  v = op(v, dpp<0x121>(v));
  if constexpr (LPT == 64) {
    V a, b;
    both<16>(v, &a, &b);
    v = op(a, b);
    both<32>(v, &a, &b);
    v = op(a, b);
  }
  return v;
}
__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
template <int LPT, typename V>
__device__ __forceinline__ V reduce_max(V v) {
  return reduce<LPT>(v, [](V a, V b) { return larger(a, b); });
}
template <int LPT>
__device__ __forceinline__ int reduce_min(int v) {
  return reduce<LPT>(v, [](int a, int b) { return min(a, b); });
}
template <int LPT, typename V>
__device__ __forceinline__ V reduce_sum(V v) {
  return reduce<LPT>(v, [](V a, V b) { return a + b; });
}

__device__ __forceinline__ double score64(int score, float l, float top) {
  return score == MOE_EP_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top);
}

// One token per LPT lanes, expert e = v * LPT + lane in register v; lane j of
// the token gets slot j's id and weight.  The selection is top_k rounds of a
// maximum over the lanes, then the lowest index among the lanes that hold it.
// Without a bias or groups the choice is the logit itself: it orders the
// experts as the score does, without the ties of a saturated score.  Otherwise
// it is the score in float64 (V = double), so that a near-tie is decided by
// the values and not by a float32 rounding.  Weights are computed in float64
// by one lane per slot and rounded once.
//
// A token costs some 60 instructions a round, so few tokens are bound by
// latency (one load, top_k rounds, one exponential) and many by issue: 16
// lanes to a token then do four tokens with the instructions of one.
//
// GROUPS (LPT 64): the token's wave has room for its choices at cs.
template <typename V, int LPT, int VPL, bool GROUPS>
__device__ __forceinline__ void route_token(const RouteKArgs& a, int64_t t, double* cs, int* id_out,
                                            float* weight_out) {
  constexpr bool kScores = std::is_same<V, double>::value;
  const int E = a.num_experts;
  const int lane = threadIdx.x & 63, sub = lane & (LPT - 1);
  const int64_t row = t * a.logits_stride;
  // without a bias and groups the logit is the choice
  const bool scores = kScores && (a.bias != nullptr || a.num_groups > 1);

  float l[VPL], bias[kScores ? VPL : 1];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = v * LPT + sub, at = e < E ? e : E - 1;
    l[v] = load_logit(a.logits, row + at, a.logits_dtype);
    if constexpr (kScores) bias[v] = a.bias ? a.bias[at] : 0.0f;
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) l[v] = v * LPT + sub < E ? clean_logit(l[v]) : -INFINITY;

  V c[VPL];
  float top = 0.0f;
  double total = 1.0;
  if (scores) {
    if constexpr (kScores) {
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
#pragma unroll
        for (int v = 0; v < VPL; ++v) c[v] /= total;
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) c[v] = score64(MOE_EP_SCORE_SIGMOID, l[v], 0.0f);
      }
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const double x = c[v] + (double)bias[v];
        c[v] = l[v] > -INFINITY && x > -INFINITY ? x : -INFINITY;   // a NaN bias closes too
      }
      if (GROUPS && a.num_groups > 1) {
        // LPT is 64 here, one token per wave: the choices go through LDS so that
        // `per` lanes side by side read a group's.
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const int e = v * LPT + sub;
          if (e < E) cs[e] = c[v];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const int G = a.num_groups, size = E / G;
        const int per = 64 >> (32 - __builtin_clz(G - 1));     // lanes to a group, a power of two
        const int group = sub / per;
        double b1 = -INFINITY, b2 = -INFINITY;
        if (group < G) {
          for (int i = sub % per; i < size; i += per) {
            const double x = cs[group * size + i];
            b2 = larger(b2, x < b1 ? x : b1);
            b1 = larger(b1, x);
          }
        }
        for (int d = 1; d < per; d *= 2) {
          const double o1 = __shfl_xor(b1, d), o2 = __shfl_xor(b2, d);
          b2 = larger(larger(b2, o2), b1 < o1 ? b1 : o1);
          b1 = larger(b1, o1);
        }
        const double value = a.group_top > 1 && b2 > -INFINITY ? b1 + b2 : b1;
        int ahead = 0;
        for (int h = 0; h < G; ++h) {
          const double o = __shfl(value, h * per);
          ahead += o > value || (o == value && h < group) ? 1 : 0;
        }
        const uint64_t open = __ballot(ahead < a.top_groups);
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const int e = v * LPT + sub;
          if (!((open >> ((e < E ? e / size : 0) * per)) & 1)) c[v] = -INFINITY;
        }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) c[v] = l[v];
  }

  int mine = INT_MAX;       // slot `sub`: its expert, and that one's logit
  float mine_l = -INFINITY;
  for (int r = 0; r < a.top_k; ++r) {
    V bv = c[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) bv = larger(bv, c[v]);
    const V best = reduce_max<LPT>(bv);
    int be = INT_MAX;
#pragma unroll
    for (int v = VPL - 1; v >= 0; --v) be = c[v] == best ? v * LPT + sub : be;
    be = best > (V)-INFINITY ? reduce_min<LPT>(be) : INT_MAX;
    float bl = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (be == v * LPT + sub) {
        c[v] = (V)-INFINITY;
        bl = l[v];
      }
    }
    if constexpr (LPT == 64) bl = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(bl), be & 63));
    else bl = __shfl(bl, (lane & ~(LPT - 1)) + (be & (LPT - 1)));
    if (!scores && r == 0) top = bl;
    if (sub == r) {
      mine = be;
      mine_l = bl;
    }
  }

  if (!scores && a.score == MOE_EP_SCORE_SOFTMAX && !a.renormalize) {
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) s += l[v] == -INFINITY ? 0.0 : score64(MOE_EP_SCORE_SOFTMAX, l[v], top);
    total = reduce_sum<LPT>(s);
  }
  const bool open = mine != INT_MAX && sub < a.top_k;
  const double s = open ? score64(a.score, mine_l, top) : 0.0;
  const double z = a.renormalize ? reduce_sum<LPT>(s) : total;
  *id_out = open ? mine : a.invalid_id;
  *weight_out = z > 0.0 ? (float)(s / z * (double)a.scale) : 0.0f;
}

}  // namespace
}  // namespace moe_ep_detail
