// gfx950 kernels of the experts' products: the linear product (rows_kernel),
// the two kernels of a whole mixture-of-experts layer for a few tokens
// (rows_kernel with the gated epilogue, then down_kernel), and the same for
// many tokens to an expert (wide_kernel, then sum_kernel).
//
// At decode sizes an expert sees a handful of tokens, so its matrices are
// read once for little arithmetic: the products are bound by streaming the
// weights from HBM.  The kernels give a wave 16 weight rows as the A operand
// of v_mfma_f32_16x16x32 and up to 16 tokens as the columns of B; waves that
// share rows split the sum over k and add their float32 accumulators through
// LDS in a fixed order, so results do not depend on timing.
//
// 4-bit weights: W[n,k] = (q - 8) * scale[n, k / g].  A byte 0000qqqq read as
// e4m3 is the subnormal q * 2^-9, so v_cvt_scalef32_pk_{bf16,f16}_fp8 with
// scale 512 turns two nibbles into two exact 16-bit integers.  The -8 comes
// from one more matrix instruction with a constant operand, and the group's
// scale multiplies the float32 partial sum: no weight is rounded.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "moe_experts_device.h"
#include "moe_experts_internal.h"
#include "moe_route_device.h"

namespace moe_ep_detail {
namespace {

// Global memory, said to the compiler: a pointer whose origin it cannot see
// would be read with flat loads, which also count as LDS accesses and make
// every wait a wait for all loads.
template <typename V>
__device__ __forceinline__ V gload(const void* p) {
  return *reinterpret_cast<const __attribute__((address_space(1))) V*>(reinterpret_cast<uintptr_t>(p));
}

// A value that is the same in all lanes, as a scalar (the compiler divides in
// vector registers).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A 16-byte load of 16-bit elements from any element address (gfx950 takes
// unaligned global loads; aligned ones cost nothing extra).
struct __attribute__((packed, aligned(2))) Elems8 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 load8(const void* p) {
  return reinterpret_cast<const __attribute__((address_space(1))) Elems8*>(reinterpret_cast<uintptr_t>(p))->v;
}
// Eight elements of a row of which only `have` exist (none: <= 0).  v was
// loaded so as to end with the row: the existing ones are its last.
__device__ __forceinline__ u32x4 cut8(const u32x4& v, int have) {
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  const u64x2 w = __builtin_bit_cast(u64x2, v);
  const int gone = 16 * (8 - max(min(have, 8), 0));     // bits
  u64x2 r;
  r[0] = gone == 0 ? w[0] : gone < 64 ? w[0] >> gone | w[1] << (64 - gone) : gone < 128 ? w[1] >> (gone - 64) : 0;
  r[1] = gone < 64 ? w[1] >> gone : 0;
  return __builtin_bit_cast(u32x4, r);
}

// How many columns (k) a step covers.
template <bool W4> struct Step;
template <> struct Step<false> { static constexpr int kCols = 64; };
template <> struct Step<true> { static constexpr int kCols = 128; };

// Where a wave finds 16 weight rows that start at row `first`: bases that are
// the same for all lanes (kept in scalar registers) and each lane's 32-bit
// byte offset from them.
template <bool W4>
struct RowPtr {
  const uint8_t* a;           // A rows
  uint32_t a_off;             // the lane's row and k offset
  const uint16_t* sc;         // 4-bit: scales of the tile, group 0
  uint32_t sc_off, sc_off2;   // the four rows with the lane's first accumulator row, and the next four
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
  const u32x2 v = gload<u32x2>(p + off);
  if constexpr (!SHIFT) {
    return v;
  } else {
    const uint64_t next = gload<uint64_t>(p + off2);
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

// The type of the matrix instruction's operands: the activations' parts are
// bfloat16 whatever the weights are (4-bit integers are exact in it too, and
// float16 weights go in as two bfloat16 each).
template <class T, int P>
using Operand = std::conditional_t<P == kParts, BF16, T>;
// Dense weights that go in as two operands.
template <class T, int G, int P>
constexpr bool kTwoPartA = G == 0 && P == kParts && std::is_same<T, F16>::value;

// acc += a (and a2) times the P parts of b.
template <class T, int G, int P>
__device__ __forceinline__ f32x4 dense_mfma(const u32x4& a, const u32x4& a2, const u32x4 (&b)[P], f32x4 acc) {
#pragma unroll
  for (int pl = 0; pl < P; ++pl) {
    acc = Operand<T, P>::mfma(a, b[pl], acc);
    if (kTwoPartA<T, G, P>) acc = Operand<T, P>::mfma(a2, b[pl], acc);
  }
  return acc;
}

// One wave's products of TL tiles of 16 weight rows with up to kCols columns
// of B, one item after another.  An item is count steps s0, s0 + ds, ...; P
// planes of B (an activation's parts) are `plane` elements apart.
//
// aim() points the loads at an item, prime() sends out its first kDepth
// steps' loads, run() goes through the steps, each step's loads kDepth steps
// ahead, and in its last steps sends out the next item's, so that the stream
// of weights never stops.  Loads return in the order they were sent, so A and
// B of a step go out together: were B sent later, the wait for it would be a
// wait for all of A's loads before it.  For the same reason no branch with a
// load stands between a load and its use: where paths join, the wait for a
// load becomes a wait for all.
//
// Only kCols of the matrix instruction's 16 columns are loaded, one 16-byte
// load a lane: as operands they would hold four times the registers, and the
// weights' prefetch needs those.  At its use a step of B goes through the
// wave's own piece of LDS, which hands it out as operands; the lanes of the
// columns beyond repeat the last one and are not stored.
//
// CUT: rows end inside a step.
template <class T, int G, bool SHIFT, bool CUT, int TL, int P>
struct Mac {
  static constexpr bool W4 = G != 0;
  static constexpr int GJ = W4 ? G / 32 : 1;              // matrix instructions per scale group
  static constexpr int kG = W4 ? 4 / GJ : 1;              // scale groups per step
  static constexpr int kStep = Step<W4>::kCols;
  static constexpr int kUnits = kStep / 8;                // 16-byte units of a column in a step
  static constexpr int kCols = 64 / kUnits;               // columns of a pass: 4 (4-bit) or 8 (dense)
  static constexpr int kPitch = P * kUnits * 16 + 16;     // bytes from column to column in LDS
  static constexpr int kLds = kCols * kPitch;             // a wave's piece
  // Dense weights leave the time to cut float32 columns into their parts on the
  // way to LDS, which are fewer bytes and registers than the parts (64 experts
  // of 4096 x 1024, 32 tokens: layer 284 us, and 302 with parts from memory);
  // 4-bit ones do not (one token's 8 experts of 7168 x 2048: 60 and 54.5 us).
  static constexpr bool kFloats = P > 1 && !W4;
  static constexpr int kB = kFloats ? 2 : P;              // 16-byte loads of a step
  typedef std::conditional_t<kFloats, float, uint16_t> Elem;
  static constexpr int kStageRegs = (W4 ? TL * (4 + 2 * kG) : TL * 8) + kB * 4;
  static constexpr int kDepth = TL == 2 ? (W4 ? 2 : 3) : (CUT ? 48 : 64) / kStageRegs;   // within 128 registers

  struct Stage {
    u32x4 a[TL][W4 ? 1 : 2];
    u32x2 sc[W4 ? TL : 1][kG];
    u32x4 b[kB];
  };
  struct Item {
    int s0, ds, count;
  };
  Stage st[kDepth];
  const uint8_t* abase[TL];
  const uint16_t* scbase[TL];
  uint32_t aoff[TL], scoff[TL], scoff2[TL];
  int shift[TL];
  const Elem* bp;             // B's row of column load_col()
  int64_t plane;
  char* lds_write;
  const char* lds_read;
  int unit8, q8;              // the lane's first element in a step's column, as loaded and as operand
  int kend, bend, full;

  // lds: the wave's piece.  bend: columns of B's rows.
  __device__ __forceinline__ void init(char* lds, const WeightK& w, int bend_, int64_t plane_) {
    const int lane = threadIdx.x & 63;
    lds_write = lds + (lane / kUnits) * kPitch + (lane % kUnits) * 16;
    lds_read = lds + min(lane & 15, kCols - 1) * kPitch + (lane >> 4) * 16;
    unit8 = lane % kUnits * 8;
    q8 = (lane >> 4) * 8;
    kend = w.cols;
    bend = bend_;
    plane = plane_;
    // steps with no column past an end of either row; at most one step follows
    full = (W4 ? bend : min(kend, bend)) / kStep;
  }
  __device__ __forceinline__ Item item(int s0, int s1, int ds) const {
    // one without steps still loads: step 0
    return s0 < s1 ? Item{s0, ds, uniform((s1 - s0 + ds - 1) / ds)} : Item{0, 0, 0};
  }
  // The column whose row this lane loads.
  static __device__ __forceinline__ int load_col() { return (threadIdx.x & 63) / kUnits; }

  __device__ __forceinline__ void load(Stage& x, int s) {
    // Past the end of a row: its last eight elements (there are eight);
    // compute() cuts them.
    const int k = CUT ? min(s * kStep + unit8, bend - 8) : s * kStep + unit8;
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      if constexpr (kFloats) x.b[i] = gload<u32x4>(bp + k + 4 * i);
      else x.b[i] = load8(bp + i * plane + k);
    }
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      if constexpr (W4) {
        x.a[t][0] = gload<u32x4>(abase[t] + (int64_t)s * 1024 + aoff[t]);
#pragma unroll
        for (int g = 0; g < kG; ++g) {          // past the end the last group's scale: it meets zeros of B
          const int group = CUT ? min(s * kG + g, (kend - 1) / (32 * GJ)) : s * kG + g;
          x.sc[t][g] = load_scales<SHIFT>(scbase[t], scoff[t], scoff2[t], shift[t], group);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = s * kStep + 32 * h;
          if constexpr (CUT) {
            const int back = max(at + q8 + 8 - kend, 0);
            x.a[t][h] = load8(abase[t] + (int64_t)at * 2 + (int32_t)(aoff[t] - back * 2));
          } else {
            x.a[t][h] = load8(abase[t] + (int64_t)at * 2 + aoff[t]);
          }
        }
      }
    }
  }

  __device__ __forceinline__ void aim(const RowPtr<W4> (&ap)[TL], const Elem* row) {
    bp = row;
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      abase[t] = ap[t].a;
      scbase[t] = ap[t].sc;
      aoff[t] = ap[t].a_off;
      scoff[t] = ap[t].sc_off;
      scoff2[t] = ap[t].sc_off2;
      shift[t] = ap[t].sc_shift;
      // Bases in scalar registers, offsets in one vector register each: left
      // alone, the compiler keeps a 64-bit vector address per load.
      asm volatile("" : "+s"(abase[t]), "+v"(aoff[t]));
      if constexpr (W4) asm volatile("" : "+s"(scbase[t]), "+v"(scoff[t]));
    }
    asm volatile("" : "+v"(unit8), "+v"(bp));
  }
  // s, with nothing computed from it kept across the caller's loop.
  static __device__ __forceinline__ int unhoisted(int s) {
    asm volatile("" : "+s"(s));
    return s;
  }
  __device__ __forceinline__ void prime(const Item& it) {
    const int first = unhoisted(it.s0), last = max(it.count - 1, 0);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      load(st[d], first + min(d, last) * it.ds);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  __device__ __forceinline__ void store_b(const u32x4 (&b)[P]) {
#pragma unroll
    for (int pl = 0; pl < P; ++pl) *reinterpret_cast<u32x4*>(lds_write + pl * kUnits * 16) = b[pl];
    // The wave's lanes read what its other lanes wrote: LDS operations of one
    // wave keep their order, the compiler has to as well.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  __device__ __forceinline__ u32x4 operand_b(int pl, int j) const {
    return *reinterpret_cast<const u32x4*>(lds_read + pl * kUnits * 16 + j * 64);
  }

  __device__ __forceinline__ void compute(f32x4 (&acc)[TL], const Stage& x, int s) {
    typedef Operand<T, P> O;
    const u32x4 minus8 = {O::kMinus8, O::kMinus8, O::kMinus8, O::kMinus8};
    u32x4 b[P];
    if constexpr (kFloats) {
      split_floats(x.b, b);
    } else {
#pragma unroll
      for (int pl = 0; pl < P; ++pl) b[pl] = x.b[pl];
    }
    if (CUT && s >= full) {
#pragma unroll
      for (int pl = 0; pl < P; ++pl) b[pl] = cut8(b[pl], bend - s * kStep - unit8);
    }
    store_b(b);
    if constexpr (W4) {
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        f32x4 corr = {0, 0, 0, 0}, part[TL];
        if constexpr (GJ * P <= 4) {
          // -8 times the columns' sums, then the nibbles on top of it
          u32x4 b[GJ][P];
#pragma unroll
          for (int i = 0; i < GJ; ++i) {
#pragma unroll
            for (int pl = 0; pl < P; ++pl) {
              b[i][pl] = operand_b(pl, g * GJ + i);
              corr = O::mfma(minus8, b[i][pl], corr);
            }
          }
#pragma unroll
          for (int t = 0; t < TL; ++t) part[t] = corr;
#pragma unroll
          for (int i = 0; i < GJ; ++i) {
#pragma unroll
            for (int t = 0; t < TL; ++t) {
              const u32x4 f = decode<O>(x.a[t][0][g * GJ + i]);
#pragma unroll
              for (int pl = 0; pl < P; ++pl) part[t] = O::mfma(f, b[i][pl], part[t]);
            }
          }
        } else {
          // side by side: there are no registers for all of a group's parts
#pragma unroll
          for (int t = 0; t < TL; ++t) part[t] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < GJ; ++i) {
            u32x4 f[TL];
#pragma unroll
            for (int t = 0; t < TL; ++t) f[t] = decode<O>(x.a[t][0][g * GJ + i]);
#pragma unroll
            for (int pl = 0; pl < P; ++pl) {
              const u32x4 b = operand_b(pl, g * GJ + i);
              corr = O::mfma(minus8, b, corr);
#pragma unroll
              for (int t = 0; t < TL; ++t) part[t] = O::mfma(f[t], b, part[t]);
            }
          }
#pragma unroll
          for (int t = 0; t < TL; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) part[t][r] += corr[r];
          }
        }
#pragma unroll
        for (int t = 0; t < TL; ++t) {
          const f32x4 sc = scale_floats<T>(x.sc[t][g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(sc[r], part[t][r], acc[t][r]);
        }
        // Groups one after another: interleaved they need more registers than there are.
        if constexpr (kG > 1) __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 b[P];
#pragma unroll
        for (int pl = 0; pl < P; ++pl) b[pl] = operand_b(pl, h);
#pragma unroll
        for (int t = 0; t < TL; ++t) {
          u32x4 a = x.a[t][h], a2 = a;
          if (CUT && s >= full) a = cut8(a, kend - s * kStep - 32 * h - q8);
          if constexpr (kTwoPartA<T, G, P>) split_f16(a, &a, &a2);
          acc[t] = dense_mfma<T, G, P>(a, a2, b, acc[t]);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }

  // acc += the item that was aimed at and primed.  aim_next(): points the
  // loads at the next item and returns it; called once if more is set.
  template <class F>
  __device__ __forceinline__ void run(f32x4 (&acc)[TL], const Item& it, bool more, F aim_next) {
    int i = 0;
    const int s0 = it.s0;
    for (; i + kDepth < it.count; i += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        compute(acc, st[d], s0 + (i + d) * it.ds);
        load(st[d], s0 + min(i + d + kDepth, it.count - 1) * it.ds);
        __builtin_amdgcn_sched_barrier(0);    // loads stay ahead: the scheduler would sink them to their uses
      }
    }
    if (more) {
      const Item nx = aim_next();
      const int first = unhoisted(nx.s0), last = max(nx.count - 1, 0);
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (i + d < it.count) compute(acc, st[d], s0 + (i + d) * it.ds);
        load(st[d], first + min(d, last) * nx.ds);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (i + d < it.count) compute(acc, st[d], s0 + (i + d) * it.ds);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
};

constexpr int kThreads = kExpertWaves * 64;

template <class T>
__device__ __forceinline__ void store_out(void* out, int64_t i, float v, int f32) {
  if (f32) static_cast<float*>(out)[i] = v;
  else static_cast<uint16_t*>(out)[i] = T::from_float(v);
}

// The pairs (token, top-k slot) that name an expert, in ascending order and
// each token once: list[i] = token << 6 | slot.  Called by a whole workgroup.
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(4))) Ints4 {
  i32x4 v;
};

template <int W>                         // waves of the workgroup
struct Lister {
  static constexpr int kUnroll = 4;     // loads in flight per thread
  int count[kUnroll][W];
  int repeated;                         // a token names the expert twice

  // At most 64 pairs, whose ids each wave holds one a lane: every wave lists
  // them for itself (they all write the same list).
  __device__ __forceinline__ int run_few(int v, int pairs, int top_k, int id, int* list) {
    const int lane = threadIdx.x & 63;
    const bool hit = lane < pairs && v == id;
    const uint64_t named = __ballot(hit);
    const int tok = (int)((uint32_t)lane / (uint32_t)top_k), slot = lane - tok * top_k;
    const bool first = hit && ((named >> (lane - slot)) & ((1ull << slot) - 1)) == 0;
    const uint64_t mask = __ballot(first);
    if (lane == 0) repeated = mask != named;
    if (first) list[__popcll(mask & ((1ull << lane) - 1))] = tok << 6 | slot;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    return __popcll(mask);
  }

  // Any number of pairs.  More than one round of run_by_one: 16 a thread at a
  // time (8192 pairs, four waves: two rounds for eight); where a token names the
  // expert twice then (rare), or more pairs name it than there are tokens, the
  // list is made again by run_by_one.
  __device__ __forceinline__ int run(const int32_t* ids, int pairs, int top_k, int id, int* list) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint64_t below = (1ull << lane) - 1;
    int m = 0;
    if (tid == 0) repeated = 0;
    if (pairs <= W * 64 * kUnroll) return run_by_one(ids, pairs, top_k, id, list);
    for (int base = 0; base < pairs; base += W * 64 * 4 * kUnroll) {
      int v[kUnroll][4];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int p = base + (u * W * 64 + tid) * 4;
        if (p + 4 <= pairs) {
          const i32x4 w = reinterpret_cast<const Ints4*>(ids + p)->v;
#pragma unroll
          for (int c = 0; c < 4; ++c) v[u][c] = w[c];
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) v[u][c] = ids[min(p + c, pairs - 1)];
        }
      }
      __syncthreads();
      int ahead[kUnroll];             // hits of lower lanes
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int p = base + (u * W * 64 + tid) * 4;
        int all = 0;
        ahead[u] = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[u][c] = p + c < pairs && v[u][c] == id;
          const uint64_t mask = __ballot(v[u][c]);
          all += __popcll(mask);
          ahead[u] += __popcll(mask & below);
        }
        if (lane == 0) count[u][wave] = all;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        int pos = m + ahead[u];
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int c = count[u][w];
          pos += w < wave ? c : 0;
          m += c;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (!v[u][c]) continue;
          const int p = base + (u * W * 64 + tid) * 4 + c;
          const int tok = (int)((uint32_t)p / (uint32_t)top_k);
          if (pos < kPassTokens) list[pos] = tok << 6 | (p - tok * top_k);
          ++pos;
        }
      }
    }
    __syncthreads();
    bool twice = m > kPassTokens;
    if (top_k > 1 && !twice) {
      for (int i = tid + 1; i < m; i += W * 64) twice |= list[i] >> 6 == list[i - 1] >> 6;
    }
    if (!__syncthreads_or(twice)) return m;
    return run_by_one(ids, pairs, top_k, id, list);
  }

  // One pair a thread at a time, each token once.
  __device__ __forceinline__ int run_by_one(const int32_t* ids, int pairs, int top_k, int id, int* list) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int m = 0;
    for (int base = 0; base < pairs; base += W * 64 * kUnroll) {
      int v[kUnroll], tok[kUnroll], slot[kUnroll];
      uint64_t mask[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int p = base + u * W * 64 + tid;
        v[u] = ids[p < pairs ? p : pairs - 1];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int p = base + u * W * 64 + tid;
        bool hit = p < pairs && v[u] == id;
        mask[u] = __ballot(hit);
        if (mask[u]) {
          tok[u] = (int)((uint32_t)p / (uint32_t)top_k);
          slot[u] = p - tok[u] * top_k;
          if (hit && slot[u] > 0) {       // an earlier slot of the token: in this wave's lanes, or before them
            const int here = min(slot[u], lane);
            bool dup = ((mask[u] >> (lane - here)) & ((1ull << here) - 1)) != 0;
            for (int i = here + 1; i <= slot[u]; ++i) dup |= ids[p - i] == id;
            if (dup) repeated = 1;
            hit = !dup;
          }
          mask[u] = __ballot(hit);
        }
        if (lane == 0) count[u][wave] = __popcll(mask[u]);
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        int before = m;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int c = count[u][w];
          before += w < wave ? c : 0;
          m += c;
        }
        if ((mask[u] >> lane) & 1) list[before + __popcll(mask[u] & ((1ull << lane) - 1))] = tok[u] << 6 | slot[u];
      }
    }
    __syncthreads();
    return m;
  }
};

// One pair as the layer's second kernel reads it.
struct alignas(8) PairRec {
  int pair;                             // token << 6 | slot
  float weight;
};

// Columns [c0, c1) of the rows of no expert here are zeros; written by the
// first slot's workgroups of W waves.
template <class T, int W>
__device__ __forceinline__ void zero_rows(const RowsKArgs& a, int c0, int c1) {
  const int lane = threadIdx.x & 63;
  for (int base = (threadIdx.x >> 6) * 64; base < a.n; base += W * 64) {
    const int id = a.ids[min(base + lane, a.n - 1)];
    uint64_t left = __ballot(base + lane < a.n && (id < a.offset || (int64_t)id - a.offset >= a.num_experts));
    while (left) {
      const int64_t row = base + __builtin_ctzll(left);
      left &= left - 1;
      for (int c = c0 + lane; c < c1; c += 64) store_out<T>(a.out, row * a.out_stride + c, 0.0f, a.out_f32);
    }
  }
}

// The weight of a listed pair: the sum of its token's weights for the expert.
__device__ __forceinline__ float pair_weight(const RowsKArgs& a, int pair, int expert, int repeated) {
  const int64_t row = (int64_t)(pair >> 6) * a.top_k;
  const int j0 = pair & 63;
  float weight = a.topk_weights ? a.topk_weights[row + j0] : 1.0f;
  if (repeated) {
    for (int j = j0 + 1; j < a.top_k; ++j) {
      if (a.ids[row + j] == expert + a.offset) weight += a.topk_weights ? a.topk_weights[row + j] : 1.0f;
    }
  }
  return weight;
}

// A workgroup takes one expert (blockIdx.y) and a run of tiles of 16 output
// rows (GATED: 16 gate rows and the 16 up rows beside them), a.split of its
// waves to a tile.  It lists the tokens that chose the expert and multiplies
// them 4 (4-bit) or 8 (dense) at a time.  GATED: silu(gate) * up goes to the
// workspace whole, in kParts parts, and the first workgroup of an expert
// leaves the plan down_kernel follows.
// Bound by HBM where an expert has one pass: gate and up of 64 dense experts 1024
// x 4096, 32 tokens, 195 us, 5.5 TB/s; 32 4-bit matrices 4096 x 7168 for 48 rows
// 118 us, 3.5 TB/s; one of them 7.3 us, mostly start-up.
// ROUTED (a few tokens, GATED): every workgroup makes the router's choice for
// itself, a wave for each token.  One token of 256 grouped experts takes it 5.5
// us, little less than a kernel of its own (6.4), but the launch and the wait
// between the two are saved (2 us of that layer with 4-bit weights, 53; two tokens
// of 8 small experts: 20.2 -> 17.6).
template <class T, int G, bool GATED, bool SHIFT, bool CUT, bool ROUTED>
__global__ void __launch_bounds__(kThreads, 4)
    rows_kernel(const std::conditional_t<ROUTED, RowsRoutedKArgs, RowsKArgs> a) {
  constexpr bool W4 = G != 0;
  constexpr int TL = GATED ? 2 : 1;
  __shared__ int list[kPassTokens];
  __shared__ Lister<kExpertWaves> lister;
  __shared__ float routed_weight[ROUTED ? kFewPairs : 1];
  __shared__ f32x4 red[kExpertWaves][TL][80];    // accumulator quarters 20 apart: no bank conflicts for rows
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y, k = a.top_k;
  const int split = a.split, group = uniform(kExpertWaves / split);      // waves to a tile, tiles at once
  const int part = uniform(wave % split), mine = uniform(wave / split);
  const int tiles = (a.inter + 15) >> 4;
  const int tile0 = blockIdx.x * a.tiles_per_block;
  const int tile1 = min(tile0 + a.tiles_per_block, tiles);

  typedef Mac<T, G, SHIFT, CUT, TL, 1> M;
  __shared__ __attribute__((aligned(16))) char bmem[kExpertWaves][M::kLds];
  M mac;
  mac.init(bmem[wave], a.w, a.w.cols, 0);

  // the expert of this slot, and its tokens
  int m = a.n, expert = 0;
  if (a.ids == nullptr) {
    for (int i = tid; i < a.n; i += kThreads) list[i] = i << 6;
    __syncthreads();
  } else {
    const int pairs = a.n * k;
    const bool few = ROUTED || pairs <= kFewPairs;
    int v = 0;
    if constexpr (ROUTED) {
      if (wave < a.n) {
        static_assert(sizeof(red) >= kRoutedTokens * kRoutedExperts * sizeof(double), "room for the choices");
        int id;
        float weight;
        route_token<double, 64, kRoutedExperts / 64, true>(
            a.route, wave, reinterpret_cast<double*>(&red[0][0][0]) + wave * kRoutedExperts, &id, &weight);
        if (lane < k) {
          list[wave * k + lane] = id;
          routed_weight[wave * k + lane] = weight;
        }
      }
      __syncthreads();
      v = list[min(lane, pairs - 1)];
      __syncthreads();
    } else if (few) {
      v = gload<int>(a.ids + min(lane, pairs - 1));
    }
    const int id = !a.by_pair ? a.offset + slot
                   : few ? __builtin_amdgcn_readlane(v, slot) : __builtin_amdgcn_readfirstlane(a.ids[slot]);
    const bool inside = id >= a.offset && (int64_t)id - a.offset < a.num_experts;
    expert = inside ? id - a.offset : 0;
    m = 0;
    if (inside) {
      m = few ? lister.run_few(v, pairs, k, id, list) : lister.run(a.ids, pairs, k, id, list);
      // of the pairs that name the same expert the first one's slot does the work
      if (a.by_pair && (list[0] >> 6) * k + (list[0] & 63) != slot) m = 0;
    }
  }
  m = __builtin_amdgcn_readfirstlane(m);

  const typename M::Item it = mac.item(part, (a.w.cols + Step<W4>::kCols - 1) / Step<W4>::kCols, split);
  auto aim = [&](int tile, int c0) {        // columns past the list repeat its last token and are not stored
    RowPtr<W4> ap[TL];
    const int at = min(tile, tiles - 1) * 16;
    ap[0] = row_ptr<W4>(a.w, expert, at);
    if constexpr (GATED) ap[1] = row_ptr<W4>(a.w, expert, a.inter + at);
    const int i = min(c0 + M::load_col(), m - 1);
    mac.aim(ap, a.x + (int64_t)(list[i] >> 6) * a.x_stride);
  };
  if (m > 0) {
    aim(tile0 + mine, 0);
    mac.prime(it);
  }
  if constexpr (GATED) {
    if (blockIdx.x == 0) {
      const int chunks = (a.n + kChunkTokens - 1) / kChunkTokens;
      auto start = [&](int c) {         // the first list entry of chunk c
        int lo = 0, hi = m;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if ((list[mid] >> 6) < c * kChunkTokens) lo = mid + 1;
          else hi = mid;
        }
        return lo;
      };
      if (tid < chunks) {
        const int o0 = start(tid), o1 = start(tid + 1);
        a.plan.head[tid * a.plan.slots + slot] = pack_head(o1 - o0, o0, expert);
      }
      PairRec* rec = reinterpret_cast<PairRec*>(a.plan.pair) + (int64_t)slot * a.n;
      for (int i = tid; i < m; i += kThreads) {
        const int at = list[i];
        float weight;
        if constexpr (ROUTED) weight = routed_weight[(at >> 6) * k + (at & 63)];     // (no expert twice to a token)
        else weight = pair_weight(a, at, expert, lister.repeated);
        rec[i] = PairRec{at, weight};
      }
    }
  } else if (a.ids != nullptr && slot == 0) {
    zero_rows<T, kExpertWaves>(a, tile0 * 16, min(tile1 * 16, a.inter));
  }
  if (m == 0) return;

  for (int t0 = tile0, c0 = 0; t0 < tile1;) {
    int t2 = t0, c2 = c0 + M::kCols;        // the item after this one
    if (c2 >= m) {
      c2 = 0;
      t2 += group;
    }
    f32x4 acc[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) acc[t] = f32x4{0, 0, 0, 0};
    mac.run(acc, it, t2 < tile1, [&]() {
      aim(t2 + mine, c2);
      return it;
    });
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TL; ++t) red[wave][t][(lane >> 4) * 20 + (lane & 15)] = acc[t];
    __syncthreads();
    const int left = min(m - c0, M::kCols);
    for (int i = tid; i < group * 256; i += kThreads) {
      const int g = i >> 8, col = (i >> 4) & 15, row = i & 15, tile = t0 + g;
      if (col >= left || tile >= tile1) continue;
      float v[TL];
#pragma unroll
      for (int t = 0; t < TL; ++t) {
        v[t] = 0.0f;
#pragma unroll
        for (int w = 0; w < kExpertWaves; ++w) {
          if (w < split) v[t] += red[g * split + w][t][(row >> 2) * 20 + col][row & 3];
        }
      }
      const int n = tile * 16 + row, at = list[c0 + col], token = at >> 6;
      if constexpr (GATED) {
        // rows past the intermediate size are zeros: the down product reads whole 16-row tiles
        const float act = n < a.inter ? v[0] / (1.0f + expf(-v[0])) * v[TL - 1] : 0.0f;
        const int64_t o = ((int64_t)token * k + (at & 63)) * a.plan.act_stride + n;
        if (a.plan.act_plane == 0) {
          static_cast<float*>(a.plan.act)[o] = act;
        } else {
          uint16_t v16[kParts];
          split_parts(act, v16);
#pragma unroll
          for (int pl = 0; pl < kParts; ++pl) static_cast<uint16_t*>(a.plan.act)[pl * a.plan.act_plane + o] = v16[pl];
        }
      } else if (n < a.inter) {
        store_out<T>(a.out, (int64_t)token * a.out_stride + n, v[0], a.out_f32);
      }
    }
    t0 = t2;
    c0 = c2;
  }
}

// A workgroup takes one tile of 16 output columns and one chunk of up to 128
// tokens, and goes through every expert that the chunk uses: their (expert,
// k step) pairs in slot order, cut into one equal run per wave.  A wave adds
// weight * product into its own copy of the chunk's output tile in LDS (each
// token at most once per expert, so lanes never meet), and the copies are
// added in wave order at the end.
// Bound by HBM: 64 dense experts 4096 x 1024, 32 tokens, 104 us, 5.1 TB/s; one
// token's 8 4-bit experts 7168 x 2048 24 us, 2.5 TB/s, a fifth of it start-up and
// three steps of loads ahead, not four, for the activations' parts (21.4 us with two
// parts).
template <class T, int G, bool CUT>
__global__ void __launch_bounds__(kThreads, 4) down_kernel(const DownKArgs a) {
  constexpr bool W4 = G != 0;
  typedef Mac<T, G, false, CUT, 1, kParts> M;
  __shared__ __attribute__((aligned(16))) char bmem[kExpertWaves][M::kLds];
  __shared__ int heads[MOE_EP_MAX_EXPERTS];
  __shared__ short slots[MOE_EP_MAX_EXPERTS];
  __shared__ int wave_count[kExpertWaves];
  extern __shared__ __attribute__((aligned(16))) float sums[];   // [wave][token of the chunk][16]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroups go round the 8 XCDs in turn: the chunks of one tile follow one
  // another on one XCD, where they find the tile's weights in its L2.
  const int xcd = blockIdx.x & 7, seq = blockIdx.x >> 3;
  const int chunk = uniform(seq % a.chunks), tile = uniform(seq / a.chunks) * 8 + xcd;
  if (tile >= a.tiles) return;
  const int t0 = chunk * kChunkTokens;
  const int nc = min(a.n - t0, kChunkTokens);
  const PlanK& p = a.plan;

  int used = 0;                     // slots with tokens in this chunk
  for (int base = 0; base < p.slots; base += kThreads) {
    const int s = base + tid;
    const int head = s < p.slots ? p.head[chunk * p.slots + s] : 0;
    const bool have = head_count(head) > 0;
    const uint64_t mask = __ballot(have);
    if (base) __syncthreads();
    if (lane == 0) wave_count[wave] = __popcll(mask);
    __syncthreads();
    int pos = used + __popcll(mask & ((1ull << lane) - 1));
#pragma unroll
    for (int w = 0; w < kExpertWaves; ++w) {
      const int c = wave_count[w];
      pos += w < wave ? c : 0;
      used += c;
    }
    if (have) {
      heads[pos] = head;
      slots[pos] = (short)s;
    }
  }
  for (int i = tid; i < kExpertWaves * nc * 16; i += kThreads) sums[i] = 0.0f;
  __syncthreads();

  used = __builtin_amdgcn_readfirstlane(used);
  float* mine = sums + wave * nc * 16;
  const int steps = (a.w.cols + Step<W4>::kCols - 1) / Step<W4>::kCols;
  const int64_t all = (int64_t)used * steps;
  int s = uniform((int)(all * wave / kExpertWaves));
  const int end = uniform((int)(all * (wave + 1) / kExpertWaves));

  // One product of the run: an expert's k steps [k0, k1) with a pass of its tokens.
  struct Item {
    int expert, k0, k1, left;
    PairRec rec;
  };
  int col0 = 0;
  auto next = [&](Item& it) -> bool {
    if (s >= end) return false;
    const int i = uniform(s / steps);
    const int head = __builtin_amdgcn_readfirstlane(heads[i]), slot = __builtin_amdgcn_readfirstlane((int)slots[i]);
    const int m = head_count(head);
    it.expert = head_expert(head);
    it.k0 = s - i * steps;
    it.k1 = min(steps, it.k0 + end - s);
    it.left = min(m - col0, M::kCols);
    const int at = head_start(head) + min(col0 + (lane & 15), m - 1);
    const u32x2 rec = gload<u32x2>(static_cast<const PairRec*>(p.pair) + (int64_t)slot * a.n + at);
    it.rec = PairRec{(int)rec[0], __uint_as_float(rec[1])};
    col0 += M::kCols;
    if (col0 >= m) {
      col0 = 0;
      s += it.k1 - it.k0;
    }
    return true;
  };
  M mac;
  mac.init(bmem[wave], a.w, p.act_stride, p.act_plane);
  auto aim = [&](const Item& it) {
    const RowPtr<W4> ap[1] = {row_ptr<W4>(a.w, it.expert, tile * 16)};
    // lane c < kCols has column c's record; the lanes that load the column need it
    const int pair = __shfl(it.rec.pair, M::load_col());
    mac.aim(ap, static_cast<const typename M::Elem*>(p.act) + ((int64_t)(pair >> 6) * a.top_k + (pair & 63)) * p.act_stride);
    return mac.item(it.k0, it.k1, 1);
  };
  Item cur;
  typename M::Item now;
  bool have = next(cur);
  if (have) {
    now = aim(cur);
    mac.prime(now);
  }
  while (have) {
    Item after;
    const bool more = next(after);
    f32x4 acc[1] = {{0, 0, 0, 0}};
    typename M::Item then = now;
    mac.run(acc, now, more, [&]() { return then = aim(after); });
    if ((lane & 15) < cur.left) {
      f32x4* o = reinterpret_cast<f32x4*>(mine + ((cur.rec.pair >> 6) - t0) * 16 + (lane >> 4) * 4);
      f32x4 v = *o;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += cur.rec.weight * acc[0][r];
      *o = v;
    }
    cur = after;
    now = then;
    have = more;
  }
  __syncthreads();
  for (int i = tid; i < nc * 16; i += kThreads) {
    const int col = tile * 16 + (i & 15);
    if (col >= a.w.rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kExpertWaves; ++w) v += sums[w * nc * 16 + i];
    store_out<T>(a.out, (int64_t)(t0 + (i >> 4)) * a.out_stride + col, v, a.out_f32);
  }
}

// ---- many tokens to an expert ------------------------------------------------

constexpr int kWideThreads = kWideWaves * 64;

// Most tiles of 16 columns in a pass: 48 columns leave registers for three
// workgroups on a compute unit, 64 for two (gate and up of 32 experts, 4096 x
// 7168, 4 bits, 32 tokens each: 208 and 212 us).
constexpr int kWideTiles = 3;

// What a wide workgroup computes.
enum WideOp { kWideLinear, kWideGated, kWideDown };

// One pass of a workgroup: kWideWaves * TL tiles of 16 weight rows, TL to a
// wave over all of k, times 16 CT columns of B.  All waves need the same B:
// each step of it is loaded once by the whole workgroup and handed out through
// LDS, in two buffers with one barrier a step.  A and B go out kDepth steps
// ahead, as in Mac.
template <class T, int G, bool SHIFT, bool CUT, int P, int CT>
struct WideMac {
  static constexpr bool W4 = G != 0;
  static constexpr int GJ = W4 ? G / 32 : 1;
  static constexpr int kG = W4 ? 4 / GJ : 1;
  static constexpr int kStep = Step<W4>::kCols, kMac = kStep / 32;
  static constexpr int TL = 2;
  static constexpr int kUnits = kStep / 8;                // 16-byte units of a column in a step
  static constexpr int kPitch = P * kUnits * 16 + 16;     // bytes from column to column in LDS
  static constexpr int kBuffer = 16 * CT * kPitch;
  static constexpr int kLoads = (16 * CT * kUnits + kWideThreads - 1) / kWideThreads;   // units a thread loads, per plane
  static constexpr int kDepth = 2;

  struct Stage {
    u32x4 a[TL][W4 ? 1 : 2];
    u32x2 sc[W4 ? TL : 1][kG];
    u32x4 b[kLoads][P];
  };

  // col_row(c): B's row of column c.  Two buffers at lds.
  template <class F>
  static __device__ __forceinline__ void run(f32x4 (&acc)[TL][CT], const WeightK& w, const RowPtr<W4> (&ap)[TL],
                                             F col_row, int64_t plane, int bend, char* lds) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int q8 = (lane >> 4) * 8, unit8 = tid % kUnits * 8;
    const int kend = w.cols;
    const int full = (W4 ? bend : min(kend, bend)) / kStep;
    const int steps = (kend + kStep - 1) / kStep;
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
    const uint16_t* row[kLoads];
    char* write[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int col = (tid + i * kWideThreads) / kUnits;
      row[i] = col_row(min(col, 16 * CT - 1));
      write[i] = lds + min(col, 16 * CT - 1) * kPitch + unit8 * 2;
    }
    const char* read = lds + (lane & 15) * kPitch + q8 * 2;

    auto load = [&](Stage& x, int s) {
      const int k = CUT ? min(s * kStep + unit8, bend - 8) : s * kStep + unit8;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
#pragma unroll
        for (int pl = 0; pl < P; ++pl) x.b[i][pl] = load8(row[i] + pl * plane + k);
      }
#pragma unroll
      for (int t = 0; t < TL; ++t) {
        if constexpr (W4) {
          x.a[t][0] = gload<u32x4>(abase[t] + (int64_t)s * 1024 + aoff[t]);
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const int group = CUT ? min(s * kG + g, (kend - 1) / (32 * GJ)) : s * kG + g;
            x.sc[t][g] = load_scales<SHIFT>(scbase[t], scoff[t], ap[t].sc_off2, ap[t].sc_shift, group);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = s * kStep + 32 * h;
            const int back = CUT ? max(at + q8 + 8 - kend, 0) : 0;
            x.a[t][h] = load8(abase[t] + (int64_t)at * 2 + (int32_t)(aoff[t] - back * 2));
          }
        }
      }
    };
    auto compute = [&](const Stage& x, int s) {
      typedef Operand<T, P> O;
      const int buffer = (s & 1) * kBuffer;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
#pragma unroll
        for (int pl = 0; pl < P; ++pl) {
          u32x4 b = x.b[i][pl];
          if (CUT && s >= full) b = cut8(b, bend - s * kStep - unit8);
          *reinterpret_cast<u32x4*>(write[i] + buffer + pl * kUnits * 16) = b;
        }
      }
      // The loads in flight stay in flight: only the LDS writes have to be done.
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
      auto operand_b = [&](int ct, int pl, int j) {
        return *reinterpret_cast<const u32x4*>(read + buffer + ct * 16 * kPitch + pl * kUnits * 16 + j * 64);
      };
      if constexpr (W4) {
        const u32x4 minus8 = {O::kMinus8, O::kMinus8, O::kMinus8, O::kMinus8};
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          u32x4 f[TL][GJ];
          f32x4 sc[TL];
#pragma unroll
          for (int t = 0; t < TL; ++t) {
            sc[t] = scale_floats<T>(x.sc[t][g]);
#pragma unroll
            for (int i = 0; i < GJ; ++i) f[t][i] = decode<O>(x.a[t][0][g * GJ + i]);
          }
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            f32x4 corr = {0, 0, 0, 0}, part[TL];
            if constexpr (P == 1) {
              u32x4 b[GJ];
#pragma unroll
              for (int i = 0; i < GJ; ++i) {
                b[i] = operand_b(ct, 0, g * GJ + i);
                corr = O::mfma(minus8, b[i], corr);
              }
#pragma unroll
              for (int t = 0; t < TL; ++t) part[t] = corr;
#pragma unroll
              for (int i = 0; i < GJ; ++i) {
#pragma unroll
                for (int t = 0; t < TL; ++t) part[t] = O::mfma(f[t][i], b[i], part[t]);
              }
            } else {
#pragma unroll
              for (int t = 0; t < TL; ++t) part[t] = f32x4{0, 0, 0, 0};
#pragma unroll
              for (int i = 0; i < GJ; ++i) {
#pragma unroll
                for (int pl = 0; pl < P; ++pl) {
                  const u32x4 b = operand_b(ct, pl, g * GJ + i);
                  corr = O::mfma(minus8, b, corr);
#pragma unroll
                  for (int t = 0; t < TL; ++t) part[t] = O::mfma(f[t][i], b, part[t]);
                }
              }
#pragma unroll
              for (int t = 0; t < TL; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) part[t][r] += corr[r];
              }
            }
#pragma unroll
            for (int t = 0; t < TL; ++t) {
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[t][ct][r] = __builtin_fmaf(sc[t][r], part[t][r], acc[t][ct][r]);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        u32x4 f[TL][2], f2[TL][2];
#pragma unroll
        for (int t = 0; t < TL; ++t) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f[t][h] = x.a[t][h];
            if (CUT && s >= full) f[t][h] = cut8(f[t][h], kend - s * kStep - 32 * h - q8);
            if constexpr (kTwoPartA<T, G, P>) split_f16(f[t][h], &f[t][h], &f2[t][h]);
            else f2[t][h] = f[t][h];
          }
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u32x4 b[P];
#pragma unroll
            for (int pl = 0; pl < P; ++pl) b[pl] = operand_b(ct, pl, h);
#pragma unroll
            for (int t = 0; t < TL; ++t) acc[t][ct] = dense_mfma<T, G, P>(f[t][h], f2[t][h], b, acc[t][ct]);
          }
        }
      }
    };
    Stage st[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      load(st[d], min(d, steps - 1));
      __builtin_amdgcn_sched_barrier(0);      // one step's loads after another's, as in the loop
    }
    for (int s = 0; s < steps; s += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (s + d < steps) compute(st[d], s + d);
        load(st[d], min(s + d + kDepth, steps - 1));      // past the last step: again, unused
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();      // the buffers are free for the next pass
  }
};

// Four elements of a row, `have` of which exist; whole: rows and their starts
// are on multiples of four elements.
template <class T>
__device__ __forceinline__ void store4(void* out, int64_t i, const f32x4& v, int f32, int have, bool whole) {
  if (whole && have >= 4) {
    if (f32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i) = v;
    } else {
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) =
          u32x2{T::from_float(v[0]) | (uint32_t)T::from_float(v[1]) << 16,
                T::from_float(v[2]) | (uint32_t)T::from_float(v[3]) << 16};
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (r < have) store_out<T>(out, i + r, v[r], f32);
  }
}
__device__ __forceinline__ bool whole_rows(const RowsKArgs& a) {
  return ((reinterpret_cast<uintptr_t>(a.out) / (a.out_f32 ? 4 : 2)) | (uintptr_t)a.out_stride) % 4 == 0;
}

// The expert with the rank-th most pairs among num_experts (at most
// kWideThreads), the lower one first among equals.  Called by a whole wide
// workgroup; counts has room for them.
__device__ __forceinline__ int busiest(const RowsKArgs& a, int rank, int* counts) {
  __shared__ int found;
  const int tid = threadIdx.x, pairs = a.n * a.top_k;
  counts[tid] = 0;
  __syncthreads();
  constexpr int kUnroll = 4;
  for (int base = 0; base < pairs; base += kWideThreads * 4 * kUnroll) {
    i32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + (u * kWideThreads + tid) * 4;
      v[u] = i32x4{-1, -1, -1, -1};       // (offset >= 0)
      if (i + 4 <= pairs) {
        v[u] = reinterpret_cast<const Ints4*>(a.ids + i)->v;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (i + c < pairs) v[u][c] = a.ids[i + c];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (v[u][c] >= a.offset && (int64_t)v[u][c] - a.offset < a.num_experts) atomicAdd(&counts[v[u][c] - a.offset], 1);
      }
    }
  }
  __syncthreads();
  if (tid < a.num_experts) {
    const int mine = counts[tid];
    int ahead = 0;
    for (int e = 0; e < a.num_experts; ++e) ahead += counts[e] > mine || (counts[e] == mine && e < tid);
    if (ahead == rank) found = tid;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(found);
}

// A workgroup takes one expert (blockIdx.y) and kWideWaves * 2 tiles of 16
// weight rows (kWideGated: as many gate as up tiles, a pair to a wave), lists
// the expert's tokens and multiplies them 48 at a time, with as many columns as
// are left in the last pass.
// kWideGated leaves its lists in the plan for kWideDown, whose workgroups are
// spared the going through all ids.
// kWideDown reads the activations of kWideGated and writes each pair's
// weighted product, in float32, for sum_kernel.
// Bound by issue: decoding, matrix and LDS instructions of a step hardly overlap
// between the waves of a workgroup, which the barrier keeps together.  32 4-bit
// experts of 4096 x 7168 and 7168 x 2048, some 1200 pairs: 197 and 190 us (1.3 to
// 2.4 TB/s of weights, an expert of 130 tokens three times), sum_kernel 15; with
// activations in two parts kWideDown would take 143.
template <class T, int G, WideOp OP, bool SHIFT, bool CUT>
__global__ void __launch_bounds__(kWideThreads, OP == kWideDown ? 2 : 3) wide_kernel(const RowsKArgs a) {
  constexpr bool W4 = G != 0;
  constexpr int TL = 2, P = OP == kWideDown ? kParts : 1, kMost = kWideTiles;
  // kWideDown's list stays in the plan: beside the activations' parts it would
  // leave room for one workgroup on a compute unit instead of two.
  __shared__ int list[OP == kWideDown ? 1 : kPassTokens];
  __shared__ Lister<kWideWaves> lister;
  __shared__ __attribute__((aligned(16))) char bmem[2 * WideMac<T, G, SHIFT, CUT, P, kMost>::kBuffer];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y, k = a.top_k;
  const int tiles = (a.inter + 15) >> 4;

  int m = a.n, expert = 0;
  const PlanK& p = a.plan;
  PairRec* rec = reinterpret_cast<PairRec*>(p.pair) + (int64_t)slot * a.n;
  if (OP == kWideDown) {
    m = p.head[slot];
    expert = __builtin_amdgcn_readfirstlane(p.head[p.slots + slot]);
  } else if (a.ids == nullptr) {
    for (int i = tid; i < a.n; i += kWideThreads) list[i] = i << 6;
    __syncthreads();
  } else {
    const int id = a.by_pair         ? __builtin_amdgcn_readfirstlane(a.ids[slot])
                   : a.busiest_first ? a.offset + busiest(a, slot, reinterpret_cast<int*>(bmem))
                                     : a.offset + slot;
    const bool inside = id >= a.offset && (int64_t)id - a.offset < a.num_experts;
    expert = inside ? id - a.offset : 0;
    m = 0;
    if (inside) {
      m = lister.run(a.ids, a.n * k, k, id, list);
      if (a.by_pair && (list[0] >> 6) * k + (list[0] & 63) != slot) m = 0;
    }
  }
  if (OP == kWideGated && blockIdx.x == 0 && blockIdx.z == 0) {
    if (tid == 0) {
      p.head[slot] = m;
      p.head[p.slots + slot] = expert;
    }
    for (int i = tid; i < m; i += kWideThreads) rec[i] = PairRec{list[i], pair_weight(a, list[i], expert, lister.repeated)};
  }
  if (OP == kWideLinear && a.ids != nullptr && slot == 0) {
    const int c0 = blockIdx.x * kWideWaves * TL * 16;
    zero_rows<T, kWideWaves>(a, c0, min(c0 + kWideWaves * TL * 16, a.inter));
  }
  m = __builtin_amdgcn_readfirstlane(m);
  if (m == 0) return;

  auto pair_at = [&](int i) { return OP == kWideDown ? gload<int>(&rec[i].pair) : list[i]; };
  const bool whole = whole_rows(a);
  RowPtr<W4> ap[TL];
  int tile[TL];           // of the output; past the last one: not stored
#pragma unroll
  for (int t = 0; t < TL; ++t) {
    tile[t] = OP == kWideGated ? blockIdx.x * kWideWaves + wave : (blockIdx.x * kWideWaves + wave) * TL + t;
    const int at = min(tile[t], tiles - 1) * 16;
    ap[t] = row_ptr<W4>(a.w, expert, OP == kWideGated && t == 1 ? a.inter + at : at);
  }
  auto pass = [&](auto ct_c, int c0) {
    constexpr int CT = decltype(ct_c)::value;
    f32x4 acc[TL][CT];
#pragma unroll
    for (int t = 0; t < TL; ++t) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) acc[t][ct] = f32x4{0, 0, 0, 0};
    }
    auto col_row = [&](int c) -> const uint16_t* {      // columns past the list repeat its last token
      const int at = pair_at(min(c0 + c, m - 1));
      if constexpr (OP == kWideDown) return static_cast<const uint16_t*>(a.plan.act) + ((int64_t)(at >> 6) * k + (at & 63)) * a.plan.act_stride;
      else return a.x + (int64_t)(at >> 6) * a.x_stride;
    };
    WideMac<T, G, SHIFT, CUT, P, CT>::run(acc, a.w, ap, col_row, a.plan.act_plane,
                                          OP == kWideDown ? a.plan.act_stride : a.w.cols, bmem);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int i = c0 + ct * 16 + (lane & 15);
      if (i >= m) continue;
      const int at = pair_at(i);
      const int64_t pair = (int64_t)(at >> 6) * k + (at & 63);
      if constexpr (OP == kWideGated) {
        if (tile[0] >= tiles) continue;
        const int n = tile[0] * 16 + (lane >> 4) * 4;
        uint16_t v16[4][kParts];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float g = acc[0][ct][r], u = acc[1][ct][r];
          // rows past the intermediate size are zeros: the down product reads whole 16-row tiles
          split_parts(n + r < a.inter ? g / (1.0f + expf(-g)) * u : 0.0f, v16[r]);
        }
        uint16_t* o = static_cast<uint16_t*>(a.plan.act) + pair * a.plan.act_stride + n;      // a multiple of four elements
#pragma unroll
        for (int pl = 0; pl < kParts; ++pl) {
          *reinterpret_cast<u32x2*>(o + pl * a.plan.act_plane) =
              u32x2{v16[0][pl] | (uint32_t)v16[1][pl] << 16, v16[2][pl] | (uint32_t)v16[3][pl] << 16};
        }
      } else {
        float weight = 1.0f;
        if constexpr (OP == kWideDown) weight = rec[i].weight;
#pragma unroll
        for (int t = 0; t < TL; ++t) {
          const int n = tile[t] * 16 + (lane >> 4) * 4;
          const int have = tile[t] < tiles ? a.inter - n : 0;
          f32x4 v = acc[t][ct];
          if constexpr (OP == kWideDown) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] *= weight;
            float* o = a.pair_out + pair * a.pair_stride + n;         // a multiple of four elements
            if (have > 0) *reinterpret_cast<f32x4*>(o) = v;           // pair_stride has room for a whole tile
          } else {
            store4<T>(a.out, (int64_t)(at >> 6) * a.out_stride + n, v, a.out_f32, have, whole);
          }
        }
      }
    }
  };
  for (int c0 = blockIdx.z * 16 * kMost; c0 < m; c0 += gridDim.z * 16 * kMost) {
    const int left = m - c0;
    if (left <= 16) pass(std::integral_constant<int, 1>{}, c0);
    else if (left <= 32) pass(std::integral_constant<int, 2>{}, c0);
    else pass(std::integral_constant<int, kMost>{}, c0);
  }
}

// out[t] = the sum of its pairs' products in slot order: those that name an
// expert here, each expert once.
template <class T>
__global__ void __launch_bounds__(256) sum_kernel(const RowsKArgs a, int hidden) {
  const int64_t t = blockIdx.y;
  const int lane = threadIdx.x & 63;
  const int id = a.ids[t * a.top_k + min(lane, a.top_k - 1)];
  bool first = lane < a.top_k && id >= a.offset && (int64_t)id - a.offset < a.num_experts;
  for (int i = 0; i < a.top_k; ++i) first &= i >= lane || __builtin_amdgcn_readlane(id, i) != id;
  const uint64_t mask = __ballot(first);        // the slots to sum
  const int h = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (h >= hidden) return;
  f32x4 v = {0, 0, 0, 0};
  for (uint64_t left = mask; left; left &= left - 1) {
    const int j = __builtin_ctzll(left);
    const f32x4 y = *reinterpret_cast<const f32x4*>(a.pair_out + (t * a.top_k + j) * a.pair_stride + h);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += y[r];
  }
  store4<T>(a.out, t * a.out_stride + h, v, a.out_f32, hidden - h, whole_rows(a));
}

// ---- launches ---------------------------------------------------------------

template <class T, int G, bool GATED, class Args>
void start_rows(Args a, hipStream_t stream) {
  constexpr bool kRouted = std::is_same<Args, RowsRoutedKArgs>::value;
  const int slots = a.ids == nullptr ? 1 : a.by_pair ? a.n * a.top_k : a.num_experts;
  const int tiles = (a.inter + 15) / 16;
  // Waves to a tile.  Eight read a dense row in pieces of 1 KiB, which DRAM
  // likes best (64 experts of 4096 x 2048, 32 tokens: 194 us; 217 at four).
  // 4-bit tiles lie in 1 KiB pieces anyway: fewer waves to a tile mean longer
  // streams and fewer sums (32 experts of 4096 x 7168: 131 us at eight, 123 at
  // four, 118 at two) while there are tiles enough for all compute units (256
  // tiles of one matrix: 7.2 us at eight, 8.8 at four).  A wave without a step
  // only waits.
  const int steps = (a.w.cols + Step<G != 0>::kCols - 1) / Step<G != 0>::kCols;
  const int64_t work = (int64_t)tiles * slots;
  a.split = kExpertWaves;
  if (G != 0 && work >= 1024) a.split = work >= 4096 ? 2 : 4;
  while (a.split > 1 && steps < a.split) a.split /= 2;
  a.tiles_per_block = kExpertWaves / a.split;
  const dim3 grid((tiles + a.tiles_per_block - 1) / a.tiles_per_block, slots);
  if constexpr (GATED && G != 0) {
    if (a.inter % 4 != 0) {               // the up rows' scales straddle their groups of four
      rows_kernel<T, G, GATED, true, true, kRouted><<<grid, kThreads, 0, stream>>>(a);
      return;
    }
  }
  if (a.w.cols % Step<G != 0>::kCols != 0)
    rows_kernel<T, G, GATED, false, true, kRouted><<<grid, kThreads, 0, stream>>>(a);
  else rows_kernel<T, G, GATED, false, false, kRouted><<<grid, kThreads, 0, stream>>>(a);
}

template <class T, int G, WideOp OP>
void start_wide(RowsKArgs a, hipStream_t stream) {
  const int slots = a.ids == nullptr ? 1 : a.by_pair ? a.n * a.top_k : a.num_experts;
  const int tiles = (a.inter + 15) / 16;
  const int per = kWideWaves * (OP == kWideGated ? 1 : 2);
  // The passes over an expert's tokens go to workgroups of their own while
  // these fill the card (they meet in L2; layer, 695 tokens of 4 of 8 experts,
  // 1784 x 200, 4 bits: 73 us, and 266 with one workgroup for all passes), as
  // many as all experts' tokens evenly spread would take.  Once the card is
  // full they would only come too late to find the weights in L2 (32 dense
  // matrices 2048 x 2048, 96 rows each: 139 us, and 103 in one workgroup).
  const int64_t blocks = (int64_t)((tiles + per - 1) / per) * slots;
  const int64_t experts = a.ids == nullptr ? 1 : a.num_experts;
  const int64_t at_once = experts * kWideTiles * 16;
  const int64_t passes = ((int64_t)a.n * a.top_k + at_once - 1) / at_once;
  const dim3 grid((tiles + per - 1) / per, slots, (unsigned)std::max<int64_t>(1, std::min(passes, 512 / blocks)));
  // The card holds some 768 workgroups at once: an expert of several passes that
  // started with the last of them would run on alone.  (32 experts of 4096 x
  // 7168 and 7168 x 2048, 4 bits, 1 to 130 of 1389 pairs each: layer 525 us in
  // the experts' order, 413 busiest first; 0 to 107 of 1147: 352 and 341.)
  // (kWideDown follows kWideGated's order, whose w.cols are its rows.)
  const int64_t then = OP == kWideGated ? ((int64_t)a.w.cols + kWideWaves * 32 - 1) / (kWideWaves * 32) * slots : 0;
  a.busiest_first = OP != kWideDown && a.ids != nullptr && !a.by_pair && std::max(blocks, then) > 512 &&
                    a.num_experts <= kWideThreads;
  if constexpr (OP == kWideGated && G != 0) {
    if (a.inter % 4 != 0) {
      wide_kernel<T, G, OP, true, true><<<grid, kWideThreads, 0, stream>>>(a);
      return;
    }
  }
  if (a.w.cols % Step<G != 0>::kCols != 0) wide_kernel<T, G, OP, false, true><<<grid, kWideThreads, 0, stream>>>(a);
  else wide_kernel<T, G, OP, false, false><<<grid, kWideThreads, 0, stream>>>(a);
}

template <class T, WideOp OP>
hipError_t start_wide(const RowsKArgs& a, int group, hipStream_t stream) {
  switch (group) {
    case 0: start_wide<T, 0, OP>(a, stream); break;
    case 32: start_wide<T, 32, OP>(a, stream); break;
    case 64: start_wide<T, 64, OP>(a, stream); break;
    default: start_wide<T, 128, OP>(a, stream); break;
  }
  return hipGetLastError();
}

template <class T>
hipError_t start_sum(const RowsKArgs& a, int hidden, hipStream_t stream) {
  const dim3 grid((hidden + 1023) / 1024, a.n);
  sum_kernel<T><<<grid, 256, 0, stream>>>(a, hidden);
  return hipGetLastError();
}

template <class T, bool GATED, class Args>
hipError_t start_rows(const Args& a, int group, hipStream_t stream) {
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
  if (a.w.cols % Step<G != 0>::kCols != 0) down_kernel<T, G, true><<<grid, kThreads, lds, stream>>>(a);
  else down_kernel<T, G, false><<<grid, kThreads, lds, stream>>>(a);
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

}  // namespace

hipError_t launch_expert_linear(const RowsKArgs& a, int dtype, int group, hipStream_t stream) {
  if (a.wide)
    return dtype == MOE_EP_BF16 ? start_wide<BF16, kWideLinear>(a, group, stream)
                                : start_wide<F16, kWideLinear>(a, group, stream);
  return dtype == MOE_EP_BF16 ? start_rows<BF16, false>(a, group, stream) : start_rows<F16, false>(a, group, stream);
}

hipError_t launch_gate_up(const RowsKArgs& a, int dtype, int group, hipStream_t stream) {
  if (a.wide)
    return dtype == MOE_EP_BF16 ? start_wide<BF16, kWideGated>(a, group, stream)
                                : start_wide<F16, kWideGated>(a, group, stream);
  return dtype == MOE_EP_BF16 ? start_rows<BF16, true>(a, group, stream) : start_rows<F16, true>(a, group, stream);
}

hipError_t launch_gate_up_routed(const RowsRoutedKArgs& a, int dtype, int group, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? start_rows<BF16, true>(a, group, stream) : start_rows<F16, true>(a, group, stream);
}

hipError_t launch_down(const DownKArgs& a, int dtype, int group, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? start_down<BF16>(a, group, stream) : start_down<F16>(a, group, stream);
}

hipError_t launch_wide_down(const RowsKArgs& a, int dtype, int group, hipStream_t stream) {
  const hipError_t e = dtype == MOE_EP_BF16 ? start_wide<BF16, kWideDown>(a, group, stream)
                                            : start_wide<F16, kWideDown>(a, group, stream);
  if (e != hipSuccess) return e;
  return dtype == MOE_EP_BF16 ? start_sum<BF16>(a, a.inter, stream) : start_sum<F16>(a, a.inter, stream);
}

}  // namespace moe_ep_detail
