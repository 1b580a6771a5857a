// gfx950 kernels of the expert-side operators: the router's selection
// (route_kernel), the experts' linear product (rows_kernel) and the two
// kernels of a whole mixture-of-experts layer for a few tokens (rows_kernel
// with the gated epilogue, then down_kernel).
//
// At decode sizes an expert sees a handful of tokens, so its matrices are
// read once for little arithmetic: the products are bound by streaming the
// weights from HBM.  Both product kernels therefore give one wave 16 weight
// rows as the A operand of v_mfma_f32_16x16x32 and up to 16 tokens as the
// columns of B; the eight waves of a workgroup share the sum over k and add
// their float32 accumulators through LDS in a fixed order, so results do not
// depend on timing.
//
// 4-bit weights: W[n,k] = (q - 8) * scale[n, k / g].  A byte 0000qqqq read as
// e4m3 is the subnormal q * 2^-9, so v_cvt_scalef32_pk_{bf16,f16}_fp8 with
// scale 512 turns two nibbles into two exact 16-bit integers.  The -8 comes
// from one more matrix instruction with a constant operand, and the group's
// scale multiplies the float32 partial sum: no weight is rounded.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

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

// ---------------------------------------------------------------------------
// route
// ---------------------------------------------------------------------------

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

// ---------------------------------------------------------------------------
// the experts' products
// ---------------------------------------------------------------------------

// A 16-byte load of 16-bit elements from any element address (gfx950 takes
// unaligned global loads; aligned ones cost nothing extra).
struct __attribute__((packed, aligned(2))) Elems8 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  return reinterpret_cast<const Elems8*>(p)->v;
}
// The same where only elements k < end of a row exist: zeros beyond.
__device__ __forceinline__ u32x4 load8_guarded(const uint16_t* p, int k, int end) {
  if (k + 8 <= end) return load8(p);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k + i < end) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  }
  return v;
}

// How many columns (k) a step covers, and matrix instructions per step.
template <bool W4> struct Step;
template <> struct Step<false> { static constexpr int kCols = 64, kMac = 2; };
template <> struct Step<true> { static constexpr int kCols = 128, kMac = 4; };

// Where a wave finds 16 weight rows that start at row `first`: bases that are
// the same for all lanes (kept in scalar registers) and each lane's 32-bit
// offset from them.
template <bool W4>
struct RowPtr {
  const uint8_t* a;           // A rows
  uint32_t a_off;             // bytes: the lane's row and k offset
  const uint16_t* sc;         // 4-bit: scales of the tile, group 0
  uint32_t sc_off, sc_off2;   // bytes: the four rows with the lane's first accumulator row, and the next four
  int sc_shift;               // bits from the first of those four rows to the lane's, the same for all lanes
};

template <bool W4>
__device__ __forceinline__ RowPtr<W4> row_ptr(const WeightK& w, int expert, int first) {
  const int lane = threadIdx.x & 63;
  const int q = lane >> 4;
  RowPtr<W4> r;
  const int row = min(first + (lane & 15), w.rows - 1);   // rows past the last repeat it
  const uint8_t* base = w.data + (int64_t)expert * w.expert_bytes;
  if constexpr (W4) {
    const int tile = first >> 4;
    r.a = base + (int64_t)tile * w.kblocks * 1024;
    r.a_off = (uint32_t)((row >> 4) - tile) * w.kblocks * 1024 + (q * 16 + (row & 15)) * 16;
    r.sc = w.scales + (int64_t)expert * w.expert_scales + (int64_t)tile * w.groups * 16;
    const int quad = (first + 4 * q) & ~3, last = (w.rows - 1) & ~3;
    const int r1 = min(quad, last), r2 = min(quad + 4, last);
    r.sc_off = ((uint32_t)((r1 >> 4) - tile) * w.groups * 16 + (r1 & 15)) * 2;
    r.sc_off2 = ((uint32_t)((r2 >> 4) - tile) * w.groups * 16 + (r2 & 15)) * 2;
    r.sc_shift = (first & 3) * 16;
  } else {
    r.a = base + (int64_t)first * w.cols * 2;
    r.a_off = ((uint32_t)(row - first) * w.cols + q * 8) * 2;
    r.sc = nullptr;
    r.sc_off = r.sc_off2 = 0;
    r.sc_shift = 0;
  }
  return r;
}

// The scales of the lane's four accumulator rows for one group: one 8-byte
// load, or (SHIFT) two and a shift where the up rows do not start on a
// multiple of four.  SHIFT waits for its loads on the spot.
template <bool SHIFT>
__device__ __forceinline__ u32x2 load_scales(const uint16_t* base, uint32_t off, uint32_t off2, int shift, int group) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base + (int64_t)group * 16);
  const u32x2 v = *reinterpret_cast<const u32x2*>(p + off);
  if constexpr (!SHIFT) {
    return v;
  } else {
    const uint64_t next = *reinterpret_cast<const uint64_t*>(p + off2);
    return __builtin_bit_cast(u32x2, __builtin_bit_cast(uint64_t, v) >> shift |
                                         (shift ? next << (64 - shift) : 0));
  }
}

template <class T>
__device__ __forceinline__ f32x4 scale_floats(const u32x2& v) {
  return f32x4{T::to_float((uint16_t)v[0]), T::to_float((uint16_t)(v[0] >> 16)), T::to_float((uint16_t)v[1]),
               T::to_float((uint16_t)(v[1] >> 16))};
}

// Eight 4-bit weights as 0..15 of the 16-bit type: the low halves of the
// word's bytes are elements 0-3, the high halves 4-7.
template <class T>
__device__ __forceinline__ u32x4 decode(uint32_t w) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  return u32x4{T::template nibbles<false>(lo), T::template nibbles<true>(lo), T::template nibbles<false>(hi),
               T::template nibbles<true>(hi)};
}

// What one step loads of the weights, two steps ahead of its use.
template <bool W4, int GJ, int TL>
struct Stage {
  static constexpr int kG = W4 ? 4 / GJ : 1;
  u32x4 a[TL][W4 ? 1 : 2];
  u32x2 sc[W4 ? TL : 1][kG];
};

// acc[tl][ct] += A(16 rows of tile tl, step columns) * B(columns of ct), over
// the steps s0, s0 + ds, ... below s1.  P planes of B (high, low part) are
// `plane` elements apart.  bend: columns of B's rows.
template <class T, bool W4, bool SHIFT, int GJ, int TL, int CT, int P>
__device__ __forceinline__ void mac(f32x4 (&acc)[TL][CT], const WeightK& w, const RowPtr<W4> (&ap)[TL],
                                    const uint16_t* const (&bp)[CT], int64_t plane, int bend, int s0, int s1,
                                    int ds) {
  constexpr int kCols = Step<W4>::kCols, kMac = Step<W4>::kMac;
  constexpr bool kStageB = CT == 1;
  constexpr int kDepth = W4 && GJ == 1 ? 2 : TL == 1 ? 4 : 2;
  typedef Stage<W4, GJ, TL> St;
  // B comes from L2: one step ahead for one column tile, at its use for more
  // (there are no registers for it).
  u32x4 bs[kStageB ? P : 1][kStageB ? kMac : 1];
  const u32x4 minus8 = {T::kMinus8, T::kMinus8, T::kMinus8, T::kMinus8};
  // Bases stay in scalar registers and offsets in one vector register each:
  // left alone, the compiler keeps a 64-bit vector address per load across
  // the caller's loop.
  const uint8_t* abase[TL];
  const uint16_t* scbase[TL];
  uint32_t aoff[TL], scoff[TL];
#pragma unroll
  for (int t = 0; t < TL; ++t) {
    abase[t] = ap[t].a;
    scbase[t] = ap[t].sc;
    aoff[t] = ap[t].a_off;
    scoff[t] = ap[t].sc_off;
    asm volatile("" : "+s"(abase[t]), "+v"(aoff[t]));
    if constexpr (W4) asm volatile("" : "+s"(scbase[t]), "+v"(scoff[t]));
  }
  const int kend = w.cols;
  // Steps with no column past an end of either row; at most one step follows.
  const int full = (W4 ? bend : (kend < bend ? kend : bend)) / kCols;

  auto load_b = [&](int ct, int pl, int j, int s) -> u32x4 {
    return load8(bp[ct] + pl * plane + (int64_t)s * kCols + 32 * j);
  };
  auto load = [&](St& st, int s) {
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      if constexpr (W4) {
        st.a[t][0] = *reinterpret_cast<const u32x4*>(abase[t] + (int64_t)s * 1024 + aoff[t]);
#pragma unroll
        for (int g = 0; g < St::kG; ++g) st.sc[t][g] = load_scales<SHIFT>(scbase[t], scoff[t], ap[t].sc_off2, ap[t].sc_shift, s * St::kG + g);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          st.a[t][h] = load8(reinterpret_cast<const uint16_t*>(abase[t] + ((int64_t)s * kCols + 32 * h) * 2 + aoff[t]));
      }
    }
  };
  auto stage_b = [&](int s) {
    if constexpr (kStageB) {
#pragma unroll
      for (int pl = 0; pl < P; ++pl) {
#pragma unroll
        for (int j = 0; j < kMac; ++j) bs[pl][j] = load_b(0, pl, j, s);
      }
    }
  };
  auto compute = [&](const St& st, int s) {
    if constexpr (W4) {
#pragma unroll
      for (int g = 0; g < St::kG; ++g) {
        f32x4 sc[TL];
        u32x4 f[TL][GJ];
#pragma unroll
        for (int t = 0; t < TL; ++t) {
          sc[t] = scale_floats<T>(st.sc[t][g]);
#pragma unroll
          for (int i = 0; i < GJ; ++i) f[t][i] = decode<T>(st.a[t][0][g * GJ + i]);
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          f32x4 corr = {0, 0, 0, 0}, part[TL];
#pragma unroll
          for (int t = 0; t < TL; ++t) part[t] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < GJ; ++i) {
#pragma unroll
            for (int pl = 0; pl < P; ++pl) {
              u32x4 b;
              if constexpr (kStageB) b = bs[pl][g * GJ + i];
              else b = load_b(ct, pl, g * GJ + i, s);
              corr = T::mfma(minus8, b, corr);
#pragma unroll
              for (int t = 0; t < TL; ++t) part[t] = T::mfma(f[t][i], b, part[t]);
            }
          }
#pragma unroll
          for (int t = 0; t < TL; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[t][ct][r] = __builtin_fmaf(sc[t][r], part[t][r] + corr[r], acc[t][ct][r]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
        for (int pl = 0; pl < P; ++pl) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u32x4 b;
            if constexpr (kStageB) b = bs[pl][h];
            else b = load_b(ct, pl, h, s);
#pragma unroll
            for (int t = 0; t < TL; ++t) acc[t][ct] = T::mfma(st.a[t][h], b, acc[t][ct]);
          }
        }
      }
    }
  };

  // The loads of a step go out kDepth steps ahead.  No branch stands between
  // a load and its use in the main loop: where paths join, the wait for a
  // load becomes a wait for all of them.
  const int last = min(s1, full);
  const int count = s0 < last ? (last - s0 + ds - 1) / ds : 0;
  if (count > 0) {
    St st[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (d < count) load(st[d], s0 + d * ds);
    }
    stage_b(s0);
    int i = 0, s = s0;
    for (; i + 2 * kDepth <= count; i += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        compute(st[d], s);
        stage_b(s + ds);
        load(st[d], s + kDepth * ds);
        s += ds;
      }
    }
#pragma unroll
    for (int d = 0; d < 2 * kDepth - 1; ++d) {
      if (i + d < count) {
        compute(st[d % kDepth], s);
        if (i + d + 1 < count) stage_b(s + ds);
        if (d < kDepth - 1 && i + d + kDepth < count) load(st[d], s + kDepth * ds);
        s += ds;
      }
    }
  }
  // The last columns, 32 at a time and element by element where a row ends.
  if (full < s1 && full >= s0 && (full - s0) % ds == 0) {
    const int q8 = ((threadIdx.x & 63) >> 4) * 8;
#pragma unroll 1
    for (int j = 0; j < kMac; ++j) {
      const int k = full * kCols + 32 * j;
      if (k >= bend) break;
      u32x4 a[TL];
      f32x4 sc[TL];
#pragma unroll
      for (int t = 0; t < TL; ++t) {
        if constexpr (W4) {
          a[t] = decode<T>(*reinterpret_cast<const uint32_t*>(ap[t].a + (int64_t)full * 1024 + ap[t].a_off + 4 * j));
          sc[t] = scale_floats<T>(load_scales<SHIFT>(scbase[t], scoff[t], ap[t].sc_off2, ap[t].sc_shift, k / (32 * GJ)));
        } else {
          a[t] = load8_guarded(reinterpret_cast<const uint16_t*>(ap[t].a + (int64_t)k * 2 + ap[t].a_off), k + q8, kend);
        }
      }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4 corr = {0, 0, 0, 0}, part[TL];
#pragma unroll
        for (int t = 0; t < TL; ++t) part[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int pl = 0; pl < P; ++pl) {
          const u32x4 b = load8_guarded(bp[ct] + pl * plane + k, k + q8, bend);
          if constexpr (W4) corr = T::mfma(minus8, b, corr);
#pragma unroll
          for (int t = 0; t < TL; ++t) part[t] = T::mfma(a[t], b, part[t]);
        }
#pragma unroll
        for (int t = 0; t < TL; ++t) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (W4) acc[t][ct][r] = __builtin_fmaf(sc[t][r], part[t][r] + corr[r], acc[t][ct][r]);
            else acc[t][ct][r] += part[t][r];
          }
        }
      }
    }
  }
}

constexpr int kThreads = kExpertWaves * 64;

// Block-wide ordered compaction: the position of this thread's item among
// the items of all threads before it, plus base.  Returns the new total.
__device__ __forceinline__ int compact(bool have, int base, int* wave_count, int* pos) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t m = __ballot(have);
  if (lane == 0) wave_count[wave] = __popcll(m);
  __syncthreads();
  int before = base, total = base;
#pragma unroll
  for (int w = 0; w < kExpertWaves; ++w) {
    const int c = wave_count[w];
    before += w < wave ? c : 0;
    total += c;
  }
  *pos = before + __popcll(m & ((1ull << lane) - 1));
  __syncthreads();
  return total;
}

__device__ __forceinline__ void store_out(void* out, int64_t i, float v, int f32, uint16_t (*round)(float)) {
  if (f32) static_cast<float*>(out)[i] = v;
  else static_cast<uint16_t*>(out)[i] = round(v);
}

// A workgroup takes one expert (blockIdx.y) and one tile of 16 output rows
// (GATED: 16 gate rows and the 16 up rows beside them).  It lists the tokens
// that chose the expert, in ascending order, and multiplies them 16 CTM at a
// time.  GATED: silu(gate) * up goes to the workspace in two 16-bit parts
// (the down product then sees it to 16 bits and more, not rounded to the 8 of
// a bfloat16), and the tile-0 workgroups leave the plan down_kernel follows.
template <class T, int G, bool GATED, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 4) rows_kernel(const RowsKArgs a) {
  constexpr bool W4 = G != 0;
  constexpr int GJ = W4 ? G / 32 : 1;
  constexpr int TL = GATED ? 2 : 1;
  __shared__ int list[kPassTokens];
  __shared__ int wave_count[kExpertWaves];
  __shared__ f32x4 red[kExpertWaves][TL][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y, tile = blockIdx.x;
  const int k = a.top_k;

  // the expert of this slot, and its tokens
  int m = 0, expert = 0;
  if (a.ids == nullptr) {
    m = a.n;
    for (int i = tid; i < a.n; i += kThreads) list[i] = i << 6;
    __syncthreads();
  } else {
    const int id = a.by_pair ? a.ids[slot] : a.offset + slot;
    const bool inside = id >= a.offset && (int64_t)id - a.offset < a.num_experts;
    expert = inside ? id - a.offset : 0;
    if (inside) {
      for (int base = 0; base < a.n; base += kThreads) {
        const int t = base + tid;
        int first = -1;
        float weight = 0.0f;
        if (t < a.n) {
          for (int j = 0; j < k; ++j) {
            if (a.ids[(int64_t)t * k + j] == id) {
              if (first < 0) first = j;
              if constexpr (GATED) weight += a.topk_weights ? a.topk_weights[(int64_t)t * k + j] : 1.0f;
            }
          }
        }
        int pos;
        m = compact(first >= 0, m, wave_count, &pos);
        if (first >= 0) {
          list[pos] = t << 6 | first;
          if constexpr (GATED) {
            if (tile == 0) {
              a.plan.pair[(int64_t)slot * a.n + pos] = t << 6 | first;
              a.plan.weight[(int64_t)slot * a.n + pos] = weight;
            }
          }
        }
      }
      __syncthreads();
      // of the pairs that name the same expert the first one's slot does the work
      if (a.by_pair && (list[0] >> 6) * k + (list[0] & 63) != slot) m = 0;
    }
  }
  if constexpr (GATED) {
    if (tile == 0) {
      if (tid == 0) a.plan.expert[slot] = expert;
      if (tid <= kMaxChunks) {          // the first list entry of each chunk of tokens
        int lo = 0, hi = m;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if ((list[mid] >> 6) < tid * kChunkTokens) lo = mid + 1;
          else hi = mid;
        }
        a.plan.off[slot * (kMaxChunks + 1) + tid] = lo;
      }
    }
  } else if (a.ids != nullptr && slot == 0) {
    // rows of no expert here: zeros, written by the first slot's workgroups
    for (int i = tid; i < a.n * 16; i += kThreads) {
      const int r = i >> 4, col = tile * 16 + (i & 15);
      const int id = a.ids[r];
      if ((id < a.offset || (int64_t)id - a.offset >= a.num_experts) && col < a.inter)
        store_out(a.out, (int64_t)r * a.out_stride + col, 0.0f, a.out_f32, T::from_float);
    }
  }
  if (m == 0) return;

  const int steps = (a.w.cols + Step<W4>::kCols - 1) / Step<W4>::kCols;
  RowPtr<W4> ap[TL];
  expert = __builtin_amdgcn_readfirstlane(expert);
  ap[0] = row_ptr<W4>(a.w, expert, tile * 16);
  if constexpr (GATED) ap[1] = row_ptr<W4>(a.w, expert, a.inter + tile * 16);

  auto run = [&](auto ct_c, int c0) {
    constexpr int CT = decltype(ct_c)::value;
    const uint16_t* bp[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {   // columns past the list repeat its last token and are not stored
      const int i = min(c0 + ct * 16 + (lane & 15), m - 1);
      bp[ct] = a.x + (int64_t)(list[i] >> 6) * a.x_stride + (lane >> 4) * 8;
    }
    f32x4 acc[TL][CT];
#pragma unroll
    for (int t = 0; t < TL; ++t) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) acc[t][ct] = f32x4{0, 0, 0, 0};
    }
    mac<T, W4, SHIFT, GJ, TL, CT, 1>(acc, a.w, ap, bp, 0, a.w.cols, wave, steps, kExpertWaves);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      __syncthreads();
#pragma unroll
      for (int t = 0; t < TL; ++t) red[wave][t][lane] = acc[t][ct];
      __syncthreads();
      const int col = tid >> 4, row = tid & 15;
      const int i = c0 + ct * 16 + col;
      if (tid < 256 && i < m) {
        float v[TL];
#pragma unroll
        for (int t = 0; t < TL; ++t) {
          v[t] = 0.0f;
#pragma unroll
          for (int w = 0; w < kExpertWaves; ++w) v[t] += red[w][t][(row >> 2) * 16 + col][row & 3];
        }
        const int n = tile * 16 + row;
        const int t = list[i] >> 6;
        if constexpr (GATED) {
          // rows past the intermediate size are zeros: the down product reads whole 16-row tiles
          const float act = n < a.inter ? v[0] / (1.0f + expf(-v[0])) * v[TL - 1] : 0.0f;
          const int64_t at = ((int64_t)t * k + (list[i] & 63)) * a.plan.act_stride + n;
          uint16_t hi, lo;
          T::split(act, &hi, &lo);
          a.plan.act[at] = hi;
          a.plan.act[a.plan.act_plane + at] = lo;
        } else if (n < a.inter) {
          store_out(a.out, (int64_t)t * a.out_stride + n, v[0], a.out_f32, T::from_float);
        }
      }
    }
  };
  for (int c0 = 0; c0 < m; c0 += 16) run(std::integral_constant<int, 1>{}, c0);
}

// A workgroup takes one tile of 16 output columns and one chunk of up to 128
// tokens, and goes through every expert that the chunk uses: their (expert,
// k step) pairs in slot order, cut into one equal run per wave.  A wave adds
// weight * product into its own copy of the chunk's output tile in LDS (each
// token at most once per expert, so lanes never meet), and the copies are
// added in wave order at the end.
template <class T, int G>
__global__ void __launch_bounds__(kThreads, 4) down_kernel(const DownKArgs a) {
  constexpr bool W4 = G != 0;
  constexpr int GJ = W4 ? G / 32 : 1;
  __shared__ int slots[MOE_EP_MAX_EXPERTS];
  __shared__ int wave_count[kExpertWaves];
  extern __shared__ __attribute__((aligned(16))) float sums[];   // [wave][token of the chunk][16]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroups go round the 8 XCDs in turn: the chunks of one tile follow one
  // another on one XCD, where they find the tile's weights in its L2.
  const int xcd = blockIdx.x & 7, seq = blockIdx.x >> 3;
  const int chunk = seq % a.chunks, tile = (seq / a.chunks) * 8 + xcd;
  if (tile >= a.tiles) return;
  const int t0 = chunk * kChunkTokens;
  const int nc = min(a.n - t0, kChunkTokens);
  const PlanK& p = a.plan;

  int used = 0;
  for (int base = 0; base < p.slots; base += kThreads) {
    const int s = base + tid;
    bool have = false;
    if (s < p.slots) {
      const int* off = p.off + s * (kMaxChunks + 1) + chunk;
      have = off[1] > off[0];
    }
    int pos;
    used = compact(have, used, wave_count, &pos);
    if (have) slots[pos] = s;
  }
  for (int i = tid; i < kExpertWaves * nc * 16; i += kThreads) sums[i] = 0.0f;
  __syncthreads();

  float* mine = sums + wave * nc * 16;
  const int steps = (a.w.cols + Step<W4>::kCols - 1) / Step<W4>::kCols;
  const int64_t all = (int64_t)used * steps;
  int64_t s = all * wave / kExpertWaves;
  const int64_t end = all * (wave + 1) / kExpertWaves;
  while (s < end) {
    const int slot = __builtin_amdgcn_readfirstlane(slots[s / steps]);
    const int k0 = (int)(s % steps);
    const int k1 = (int)min((int64_t)steps, k0 + (end - s));
    s += k1 - k0;
    const int expert = __builtin_amdgcn_readfirstlane(p.expert[slot]);
    const int* off = p.off + slot * (kMaxChunks + 1) + chunk;
    const int o0 = __builtin_amdgcn_readfirstlane(off[0]);
    const int m = __builtin_amdgcn_readfirstlane(off[1]) - o0;
    const int64_t at = (int64_t)slot * a.n + o0;
    RowPtr<W4> ap[1] = {row_ptr<W4>(a.w, expert, tile * 16)};
    auto run = [&](auto ct_c, int c0) {
      constexpr int CT = decltype(ct_c)::value;
      const uint16_t* bp[CT];
      int tok[CT];
      float weight[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const int col = c0 + ct * 16 + (lane & 15);
        const int i = min(col, m - 1);
        const int pair = p.pair[at + i];
        weight[ct] = p.weight[at + i];
        tok[ct] = col < m ? (pair >> 6) - t0 : -1;
        bp[ct] = p.act + ((int64_t)(pair >> 6) * a.top_k + (pair & 63)) * p.act_stride + (lane >> 4) * 8;
      }
      f32x4 acc[1][CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) acc[0][ct] = f32x4{0, 0, 0, 0};
      mac<T, W4, false, GJ, 1, CT, 2>(acc, a.w, ap, bp, p.act_plane, p.act_stride, k0, k1, 1);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        if (tok[ct] >= 0) {
          f32x4* o = reinterpret_cast<f32x4*>(mine + tok[ct] * 16 + (lane >> 4) * 4);
          f32x4 v = *o;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] += weight[ct] * acc[0][ct][r];
          *o = v;
        }
      }
    };
    for (int c0 = 0; c0 < m; c0 += 16) run(std::integral_constant<int, 1>{}, c0);
  }
  __syncthreads();
  for (int i = tid; i < nc * 16; i += kThreads) {
    const int col = tile * 16 + (i & 15);
    if (col >= a.w.rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kExpertWaves; ++w) v += sums[w * nc * 16 + i];
    store_out(a.out, (int64_t)(t0 + (i >> 4)) * a.out_stride + col, v, a.out_f32, T::from_float);
  }
}

template <class T, int G, bool GATED>
void start_rows(const RowsKArgs& a, hipStream_t stream) {
  const int slots = a.ids == nullptr ? 1 : a.by_pair ? a.n * a.top_k : a.num_experts;
  const dim3 grid((a.inter + 15) / 16, slots);
  if constexpr (GATED && G != 0) {
    if (a.inter % 4 != 0) {               // the up rows' scales straddle their groups of four
      rows_kernel<T, G, GATED, true><<<grid, kThreads, 0, stream>>>(a);
      return;
    }
  }
  rows_kernel<T, G, GATED, false><<<grid, kThreads, 0, stream>>>(a);
}

template <class T, bool GATED>
hipError_t start_rows(const RowsKArgs& a, int group, hipStream_t stream) {
  switch (group) {
    case 0: start_rows<T, 0, GATED>(a, stream); break;
    case 32: start_rows<T, 32, GATED>(a, stream); break;
    case 64: start_rows<T, 64, GATED>(a, stream); break;
    default: start_rows<T, 128, GATED>(a, stream); break;
  }
  return hipGetLastError();
}

template <class T, int G>
void start_down(const DownKArgs& a, hipStream_t stream) {
  const int grid = (a.tiles + 7) / 8 * 8 * a.chunks;
  const int nc = std::min(a.n, kChunkTokens);
  const size_t lds = (size_t)kExpertWaves * nc * 16 * sizeof(float);
  down_kernel<T, G><<<grid, kThreads, lds, stream>>>(a);
}

template <class T>
hipError_t start_down(const DownKArgs& a, int group, hipStream_t stream) {
  switch (group) {
    case 0: start_down<T, 0>(a, stream); break;
    case 32: start_down<T, 32>(a, stream); break;
    case 64: start_down<T, 64>(a, stream); break;
    default: start_down<T, 128>(a, stream); break;
  }
  return hipGetLastError();
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

hipError_t launch_expert_linear(const RowsKArgs& a, int dtype, int group, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? start_rows<BF16, false>(a, group, stream) : start_rows<F16, false>(a, group, stream);
}

hipError_t launch_gate_up(const RowsKArgs& a, int dtype, int group, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? start_rows<BF16, true>(a, group, stream) : start_rows<F16, true>(a, group, stream);
}

hipError_t launch_down(const DownKArgs& a, int dtype, int group, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? start_down<BF16>(a, group, stream) : start_down<F16>(a, group, stream);
}

}  // namespace moe_ep_detail
