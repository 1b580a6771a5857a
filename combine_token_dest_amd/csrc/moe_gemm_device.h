// The matrix product that the dense operators' kernels share:
//   C[q][p] = sum over k of Q(q, k) P(p, k),
// 16-bit operands, float32 sums in v_mfma_f32_32x32x16.  Either operand may
// lie with k side by side (KC: rows of k, such as x and the weights in x W^T)
// or with its rows side by side (rows of p or q, such as the weights in dy W
// and both operands of dy^T x).
//
// A workgroup makes a tile of TP x TQ results from tiles of 64 k in LDS, two
// buffers in turn: while the waves work on one, the other fills.  Each wave
// keeps its part of the results in registers.  P is the matrix instructions'
// A side, so a lane holds runs of four neighbouring p of one q: stores of
// rows of C.
//
// LDS layout, in 16-byte units of 8 elements.  KC: a row of 64 k is 8 units,
// unit u of row r at u ^ (r & 7), so that the 8 lanes that read side by side
// meet all banks.  Else: a row holds one k of all T rows, and unit u of row k
// is at u ^ 2 (k & 3); ds_read_b64_tr_b16 reads 4 k x 16 rows for 16 lanes
// (lane i the 8 bytes at k = i / 4, rows 4 (i % 4) and on) and hands lane i
// row i's four k.
//
// DIRECT: tiles go from memory to LDS without passing registers
// (global_load_lds of 16 bytes a lane), which needs rows of 16-byte alignment.
// Otherwise through registers, from any element address, with what is past
// the edges replaced by zeros; the same way goes the last tile of a k that 64
// does not divide.  Rows past the last repeat it; their results are not
// stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dense_internal.h"
#include "moe_experts_device.h"

namespace moe_ep_detail {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

#define MOE_EP_LDS __attribute__((address_space(3)))
#define MOE_EP_GLOBAL __attribute__((address_space(1)))

template <class T>
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, const f32x16& c);
template <>
__device__ __forceinline__ f32x16 mfma32<BF16>(const u32x4& a, const u32x4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
template <>
__device__ __forceinline__ f32x16 mfma32<F16>(const u32x4& a, const u32x4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                0);
}

// 16 bytes of 16-bit elements from any element address of global memory.
struct __attribute__((packed, aligned(2))) AnyHalf8 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 load_any8(const void* p) {
  return reinterpret_cast<const MOE_EP_GLOBAL AnyHalf8*>(reinterpret_cast<uintptr_t>(p))->v;
}

// Eight elements of which only the last `have` (1..7) of v exist: those, then zeros.
__device__ __forceinline__ u32x4 keep_last(const u32x4& v, int have) {
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  const u64x2 w = __builtin_bit_cast(u64x2, v);
  const int gone = 16 * (8 - have);
  u64x2 r;
  r[0] = gone < 64 ? w[0] >> gone | w[1] << (64 - gone) : w[1] >> (gone - 64);
  r[1] = gone < 64 ? w[1] >> gone : 0;
  return __builtin_bit_cast(u32x4, r);
}

constexpr int kGemmK = 64;        // k of a tile

// One operand's tile.  GATED: of its T rows, every other 32 are rows of the
// first half of the matrix (the gate) and the 32 after them the same rows of
// the second half.
template <bool KC, bool GATED, int T, int THREADS, bool DIRECT>
struct Side {
  static constexpr int kBytes = T * kGemmK * 2;
  static constexpr int kLoads = kBytes / 16 / THREADS;
  static constexpr int kReads = KC ? 1 : 2;               // LDS reads of a fragment
  static_assert(kLoads * 16 * THREADS == kBytes && (KC || T >= 64), "whole loads");

  // DIRECT: an address is base (the same for a wave) + a 32-bit offset of the
  // lane; else 64 bits, for any stride.  Tiles with k side by side step through
  // an operand's rows load by load, where the last row may repeat; the others
  // through k, a fixed distance apart.
  static constexpr int kOffsets = KC ? kLoads : 1;
  const uint8_t* base;
  uint32_t off[kOffsets];
  int64_t half;               // GATED: bytes from a gate row to its up row
  int64_t apart;              // !KC: bytes from load to load
  const uint8_t* src[kLoads]; // !DIRECT
  int64_t step;               // bytes from one tile of k to the next
  int first, rows;            // of the tile; of the operand

  static __device__ __forceinline__ int unit(int i) { return i * THREADS + (int)threadIdx.x; }
  static __device__ __forceinline__ int k_row(int i) { return unit(i) / (T / 8); }                     // !KC
  static __device__ __forceinline__ int k_unit(int i) { return (unit(i) & 7) ^ (unit(i) >> 3 & 7); }   // KC
  static __device__ __forceinline__ int col(int i) {                                                   // !KC
    const int pos = unit(i) % (T / 8);
    return (pos ^ (k_row(i) & 3) * 2) * 8;
  }
  // GATED: whether the rows of load i, the same for a wave, are up rows.
  static __device__ __forceinline__ int is_up(int i) {
    return ((i * THREADS + __builtin_amdgcn_readfirstlane(threadIdx.x)) >> 8) & 1;
  }
  // KC: the operand's row (of its half) of load i.
  __device__ __forceinline__ int row(int i) const {
    const int r = unit(i) >> 3;
    return min(first + (GATED ? (r >> 6) * 32 + (r & 31) : r), rows - 1);
  }

  __device__ __forceinline__ void aim(const MatK& m, int first_row) {
    first = first_row;
    rows = m.rows;
    step = KC ? kGemmK * 2 : m.stride * kGemmK * 2;
    half = (int64_t)m.rows * m.stride * 2;
    apart = m.stride * (THREADS * 8 / T) * 2;
    static_assert(KC || THREADS * 8 / T % 4 == 0, "a lane's column is the same in all loads");
    if constexpr (DIRECT) {
      base = reinterpret_cast<const uint8_t*>(m.p) + (KC ? (int64_t)first * m.stride : first) * 2;
      if constexpr (KC) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) off[i] = (uint32_t)((row(i) - first) * (int)m.stride + k_unit(i) * 8) * 2;
      } else {
        off[0] = (uint32_t)(k_row(0) * (int)m.stride + min(col(0), rows - 8 - first)) * 2;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int64_t at = KC ? ((int64_t)row(i) + (GATED && is_up(i) ? rows : 0)) * m.stride + k_unit(i) * 8
                              : (int64_t)k_row(i) * m.stride + first + col(i);
        src[i] = reinterpret_cast<const uint8_t*>(m.p + at);
      }
    }
  }

  __device__ __forceinline__ const uint8_t* address(int i) const {
    if constexpr (!DIRECT) return src[i];
    else if constexpr (KC) return base + (GATED && is_up(i) ? half : 0) + off[i];
    else return base + i * apart + off[0];
  }
  __device__ __forceinline__ void next() {
    if constexpr (DIRECT) {
      base += step;
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) src[i] += step;
    }
  }

  __device__ __forceinline__ void load(MOE_EP_LDS char* __restrict__ dst) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      __builtin_amdgcn_global_load_lds(
          reinterpret_cast<const MOE_EP_GLOBAL uint32_t*>(reinterpret_cast<uintptr_t>(address(i))),
          (MOE_EP_LDS uint32_t*)(dst + i * THREADS * 16 + wave * 1024), 16, 0, 0);
    next();
  }

  // The tile whose first k has `left` after it (and with it), through registers.
  __device__ __forceinline__ void fetch(u32x4 (&v)[kLoads], int left) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int have = KC ? left - k_unit(i) * 8 : (k_row(i) < left ? rows - (first + col(i)) : 0);
      if (have >= 8) {
        v[i] = load_any8(address(i));
      } else if (!DIRECT && have > 0) {
        v[i] = keep_last(load_any8(address(i) + (have - 8) * 2), have);
      } else {
        v[i] = u32x4{0, 0, 0, 0};
      }
    }
    next();
  }
  static __device__ __forceinline__ void put(MOE_EP_LDS char* __restrict__ dst, const u32x4 (&v)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) *(MOE_EP_LDS u32x4*)(dst + unit(i) * 16) = v[i];
  }

  // The operand of a matrix instruction: 32 rows from r0, 16 k from 16 ks.
  static __device__ __forceinline__ u32x4 frag(const MOE_EP_LDS char* __restrict__ s, int r0, int ks) {
    const int lane = threadIdx.x & 63;
    if constexpr (KC) {
      const int row = r0 + (lane & 31), u = ks * 2 + (lane >> 5);
      return *(const MOE_EP_LDS u32x4*)(s + row * 128 + (u ^ (row & 7)) * 16);
    } else {
      const int g = lane >> 4, i = lane & 15;
      const int k = ks * 16 + (g >> 1) * 8 + (i >> 2);
      const int row = r0 + (g & 1) * 16 + (i & 3) * 4;
      const MOE_EP_LDS char* p = s + k * (T * 2) + ((row >> 3) ^ (k & 3) * 2) * 16 + (row & 7) * 2;
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_EP_LDS s16x4*)p));
      const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_EP_LDS s16x4*)(p + 8 * T)));
      return u32x4{a[0], a[1], b[0], b[1]};
    }
  }
};

// WP x WQ waves share a tile of TP x TQ.
template <class T, bool PKC, bool QKC, bool GATED, int TP, int TQ, int WP, int WQ, bool DIRECT>
struct Gemm {
  static constexpr int kThreads = WP * WQ * 64;
  static constexpr int FP = TP / WP / 32, FQ = TQ / WQ / 32;      // a wave's fragments
  typedef Side<PKC, GATED, TP, kThreads, DIRECT> SideP;
  typedef Side<QKC, false, TQ, kThreads, DIRECT> SideQ;
  static constexpr int kBuffer = SideP::kBytes + SideQ::kBytes;
  typedef f32x16 Acc[FP][FQ];
  static_assert(!GATED || FP % 2 == 0, "a wave holds gate and up of a column");

  // Where a wave's part of the tile starts.
  static __device__ __forceinline__ int wave_p() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % WP * (TP / WP);
  }
  static __device__ __forceinline__ int wave_q() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / WP * (TQ / WQ);
  }

  static __device__ __forceinline__ void frags(const MOE_EP_LDS char* __restrict__ s, u32x4 (&p)[FP], u32x4 (&q)[FQ],
                                               int ks) {
#pragma unroll
    for (int j = 0; j < FQ; ++j) q[j] = SideQ::frag(s + SideP::kBytes, wave_q() + j * 32, ks);
#pragma unroll
    for (int i = 0; i < FP; ++i) p[i] = SideP::frag(s, wave_p() + i * 32, ks);
  }

  // One tile of k: the reads of the next 16 k go between the products of
  // these (a wave alone would wait for each fragment otherwise).
  static __device__ __forceinline__ void compute(const MOE_EP_LDS char* __restrict__ s, Acc& acc) {
    u32x4 p[2][FP], q[2][FQ];
    frags(s, p[0], q[0], 0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks < 3) frags(s, p[(ks + 1) & 1], q[(ks + 1) & 1], ks + 1);
#pragma unroll
      for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = mfma32<T>(p[ks & 1][i], q[ks & 1][j], acc[i][j]);
    }
    constexpr int kRead = 0x100, kMfma = 0x008;           // sched_group_barrier's classes
    constexpr int reads = SideP::kReads * FP + SideQ::kReads * FQ, products = FP * FQ;
    constexpr int each = (reads + products - 1) / products;
    __builtin_amdgcn_sched_group_barrier(kRead, reads, 0);
#pragma unroll
    for (int ks = 0; ks < 3; ++ks) {
#pragma unroll
      for (int i = 0; i < products; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        if (i * each < reads) __builtin_amdgcn_sched_group_barrier(kRead, each, 0);
      }
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, products, 0);
  }

  // All waves have filled this buffer, and read the other for the last time.
  static __device__ __forceinline__ void turn() {
    __builtin_amdgcn_s_waitcnt(0x0070);                   // vmcnt(0), lgkmcnt(0): loads to LDS are counted as memory's
    __syncthreads();
  }

  // A step; the next tile, of `left` k, is loaded meanwhile.  The buffers are
  // parameters of their own so that the compiler knows them apart; it would
  // wait for the loads to LDS before each read of it otherwise.
  static __device__ __forceinline__ void direct_step(const MOE_EP_LDS char* __restrict__ cur,
                                                     MOE_EP_LDS char* __restrict__ nxt, SideP& sp, SideQ& sq, Acc& acc,
                                                     int left) {
    turn();
    if (left >= kGemmK) {
      sp.load(nxt);
      sq.load(nxt + SideP::kBytes);
    } else if (left > 0) {
      fill(nxt, sp, sq, left);
    }
    __builtin_amdgcn_sched_barrier(0);
    compute(cur, acc);
  }
  static __device__ __forceinline__ void staged_step(const MOE_EP_LDS char* __restrict__ cur,
                                                     MOE_EP_LDS char* __restrict__ nxt, SideP& sp, SideQ& sq, Acc& acc,
                                                     int left) {
    __syncthreads();
    u32x4 vp[SideP::kLoads], vq[SideQ::kLoads];
    if (left > 0) {
      sp.fetch(vp, left);
      sq.fetch(vq, left);
    }
    compute(cur, acc);
    if (left > 0) {
      SideP::put(nxt, vp);
      SideQ::put(nxt + SideP::kBytes, vq);
    }
  }
  static __device__ __forceinline__ void fill(MOE_EP_LDS char* __restrict__ dst, SideP& sp, SideQ& sq, int left) {
    {
      u32x4 v[SideP::kLoads];
      sp.fetch(v, left);
      SideP::put(dst, v);
    }
    u32x4 v[SideQ::kLoads];
    sq.fetch(v, left);
    SideQ::put(dst + SideP::kBytes, v);
  }

  // The tile's sums over all K; lds holds two buffers.
  static __device__ __forceinline__ void run(MOE_EP_LDS char* lds, SideP& sp, SideQ& sq, int K, Acc& acc) {
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
      for (int j = 0; j < FQ; ++j) acc[i][j] = f32x16{};
    if (DIRECT && K >= kGemmK) {
      sp.load(lds);
      sq.load(lds + SideP::kBytes);
    } else if (K > 0) {
      fill(lds, sp, sq, K);
    }
    int cur = 0;
#pragma unroll 1
    for (int left = K; left > 0; left -= kGemmK) {
      if constexpr (DIRECT) direct_step(lds + cur, lds + (kBuffer - cur), sp, sq, acc, left - kGemmK);
      else staged_step(lds + cur, lds + (kBuffer - cur), sp, sq, acc, left - kGemmK);
      cur = kBuffer - cur;
    }
  }
};

// Which tile a workgroup makes.  Each XCD (workgroups go to the 8 of them in
// turn) takes a run of tiles, and a run goes through 8 tiles of q before the
// next p, so that what an XCD reads at one time stays in its L2.
__device__ __forceinline__ void tile_of(int ptiles, int qtiles, int* pt, int* qt) {
  const int n = gridDim.x, x = blockIdx.x % 8, i = blockIdx.x / 8, per = n / 8, rem = n % 8;
  const int b = x * per + min(x, rem) + i;
  constexpr int kGroup = 8;
  const int group = b / (kGroup * ptiles), q0 = group * kGroup, height = min(kGroup, qtiles - q0);
  const int in = b - group * kGroup * ptiles;
  *qt = q0 + in % height;
  *pt = in / height;
}

// Four neighbouring results to any element address; those past `have` are left out.
template <class T>
__device__ __forceinline__ void store4(void* out, int64_t at, bool f32, int have, const float (&v)[4]) {
  struct __attribute__((packed, aligned(2))) Two {
    u32x2 v;
  };
  struct __attribute__((packed, aligned(4))) Four {
    f32x4 v;
  };
  if (have <= 0) return;
  if (f32) {
    float* p = static_cast<float*>(out) + at;
    if (have >= 4) {
      reinterpret_cast<Four*>(p)->v = f32x4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < have) p[e] = v[e];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    uint16_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = T::from_float(v[e]);
    if (have >= 4) {
      reinterpret_cast<Two*>(p)->v = u32x2{(uint32_t)h[0] | (uint32_t)h[1] << 16, (uint32_t)h[2] | (uint32_t)h[3] << 16};
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < have) p[e] = h[e];
    }
  }
}

}  // namespace
}  // namespace moe_ep_detail
