// The matrix product that the dense operators' kernels share:
//   C[q][p] = sum over k of Q(q, k) P(p, k),
// 16-bit operands, float32 sums in v_mfma_f32_16x16x32.  Either operand may
// lie with k side by side (KC: rows of k, such as x and the weights in x W^T)
// or with its rows side by side (rows of p or q, such as the weights in dy W
// and both operands of dy^T x).
//
// A workgroup makes a tile of TP x TQ results from tiles of kK k in LDS, two
// buffers in turn: while the waves work on one, the other fills.  WP x WQ
// waves share the results, each with its part in registers, and WK such groups
// share k, whose sums are added through LDS at the end, in a fixed order: with
// few tiles a CU has one workgroup, and one wave a SIMD would wait for each of
// its LDS reads.  P is the matrix instructions' A side, so a lane holds four
// neighbouring p of one q: stores of rows of C.
//
// A large product is bound by the card's power: 8192 x 4096 x 7168 takes 300 us
// on zeros and 380 to 400 on random numbers (1.20 to 1.26 PFLOP/s; a training
// step's products with rows side by side 457 and 442).  The same tiles in
// v_mfma_f32_32x32x16 take 13% more.  Bank conflicts are 14 to 22% of the cycles
// where rows lie side by side, and 12 to 22% where a row of LDS has 128 k and
// more, which are spread over 8 units only; layouts without any take the same
// time in both (8192 rows, and 1024 rows of 7168 x 2048 at one tile a CU).
//
// LDS layout, in 16-byte units of 8 elements.  KC: a row of kK k, unit u of
// row r at u ^ (r & 7), so that the 8 lanes that read side by side meet all
// banks.  Else: a row holds one k of all T rows, and unit u of row k is at
// u ^ 2 (k & 3); ds_read_b64_tr_b16 reads 4 k x 16 rows for 16 lanes (lane i
// the 8 bytes at k = i / 4, rows 4 (i % 4) and on) and hands lane i row i's
// four k.
//
// DIRECT: tiles go from memory to LDS without passing registers
// (global_load_lds of 16 bytes a lane), which needs rows of 16-byte alignment.
// Otherwise through registers, from any element address, with what is past
// the edges replaced by zeros; the same way goes the last tile of a k that kK
// does not divide.  Rows past the last repeat it; their results are not
// stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>


#include "moe_dense_internal.h"
#include "moe_experts_device.h"
#include "moe_tile_rule.h"

namespace moe_ep_detail {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

#define MOE_EP_LDS __attribute__((address_space(3)))
#define MOE_EP_GLOBAL __attribute__((address_space(1)))

// 16 bytes of 16-bit elements from any element address of global memory.
struct __attribute__((packed, aligned(2))) AnyHalf8 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 load_any8(const void* p) {
  return reinterpret_cast<const MOE_EP_GLOBAL AnyHalf8*>(reinterpret_cast<uintptr_t>(p))->v;
}

// Eight elements of which only the last `have` (none: <= 0; all: >= 8) of v
// exist: those, then zeros.
__device__ __forceinline__ u32x4 keep_last(const u32x4& v, int have) {
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  const u64x2 w = __builtin_bit_cast(u64x2, v);
  const int gone = 16 * (8 - max(min(have, 8), 0));
  u64x2 r;
  r[0] = gone == 0 ? w[0] : gone < 64 ? w[0] >> gone | w[1] << (64 - gone) : gone < 128 ? w[1] >> (gone - 64) : 0;
  r[1] = gone < 64 ? w[1] >> gone : 0;
  return __builtin_bit_cast(u32x4, r);
}

// One operand's tile, K k of T rows.  GATED: of its rows, every other 16 are
// rows of the first half of the matrix (the gate) and the 16 after them the
// same rows of the second half.
template <bool KC, bool GATED, int T, int K, int THREADS, bool DIRECT>
struct Side {
  static constexpr int kBytes = T * K * 2;
  static constexpr int kLoads = kBytes / 16 / THREADS;
  static constexpr int kReads = KC ? 1 : 2;               // LDS reads of a fragment
  static constexpr int kUnits = (KC ? K : T) / 8;         // of a row in LDS
  static_assert(kLoads * 16 * THREADS == kBytes && kUnits >= 8, "whole loads, rows of all banks");

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
  static __device__ __forceinline__ int lds_row(int i) { return unit(i) / kUnits; }
  // KC: the first of the unit's eight k; else the first of its rows.
  static __device__ __forceinline__ int along(int i) {
    const int pos = unit(i) % kUnits, r = lds_row(i);
    return (pos ^ (KC ? r & 7 : (r & 3) * 2)) * 8;
  }
  // GATED: whether the rows of load i, the same for a wave, are up rows.
  static __device__ __forceinline__ int is_up(int i) {
    static_assert(!GATED || 64 / kUnits <= 16, "a wave's rows are of one half");
    return (i * THREADS + __builtin_amdgcn_readfirstlane(threadIdx.x)) / kUnits >> 4 & 1;
  }
  // KC: the operand's row (of its half) of load i.
  __device__ __forceinline__ int row(int i) const {
    const int r = lds_row(i);
    return min(first + (GATED ? (r >> 5) * 16 + (r & 15) : r), rows - 1);
  }

  __device__ __forceinline__ void aim(const MatK& m, int first_row) {
    first = first_row;
    rows = m.rows;
    step = KC ? K * 2 : m.stride * K * 2;
    half = (int64_t)m.rows * m.stride * 2;
    apart = m.stride * (THREADS / kUnits) * 2;
    static_assert(KC || THREADS / kUnits % 4 == 0, "a lane's rows are the same in all loads");
    if constexpr (DIRECT) {
      base = reinterpret_cast<const uint8_t*>(m.p) + (KC ? (int64_t)first * m.stride : first) * 2;
      if constexpr (KC) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) off[i] = (uint32_t)((row(i) - first) * (int)m.stride + along(i)) * 2;
      } else {
        off[0] = (uint32_t)(lds_row(0) * (int)m.stride + min(along(0), rows - 8 - first)) * 2;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int64_t at = KC ? ((int64_t)row(i) + (GATED && is_up(i) ? rows : 0)) * m.stride + along(i)
                              : (int64_t)lds_row(i) * m.stride + first + along(i);
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

  // By so many elements.
  __device__ __forceinline__ void move(int64_t elements) {
    if constexpr (DIRECT) {
      base += elements * 2;
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) src[i] += elements * 2;
    }
  }

  // Past the next `count` tiles of k (below 0: back over the last).
  __device__ __forceinline__ void skip(int count) {
    if constexpr (DIRECT) {
      base += count * step;
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) src[i] += count * step;
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

  // The tile whose first k has `left` (at least 1) after it (and with it),
  // through registers.  At an edge a unit that ends past it is loaded so as to
  // end there, and moved: with a branch for each unit its load would wait for
  // the one before.
  __device__ __forceinline__ void fetch(u32x4 (&v)[kLoads], int left) {
    if (left >= K && (KC || first + T <= rows)) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) v[i] = load_any8(address(i));
    } else {
      int have[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        have[i] = (KC ? left : rows - first) - along(i);
        int64_t back = (int64_t)(min(have[i], 8) - 8) * 2;
        // DIRECT: units past the last row's are loaded from it already
        if (!KC && DIRECT) back = 0;
        if (!KC) back -= max(lds_row(i) - (left - 1), 0) * (step / K);
        v[i] = load_any8(address(i) + back);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) v[i] = keep_last(v[i], KC || lds_row(i) < left ? have[i] : 0);
    }
    next();
  }
  static __device__ __forceinline__ void put(MOE_EP_LDS char* __restrict__ dst, const u32x4 (&v)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) *(MOE_EP_LDS u32x4*)(dst + unit(i) * 16) = v[i];
  }

  // The operand of a matrix instruction: 16 rows from r0, 32 k from 32 ks.
  static __device__ __forceinline__ u32x4 frag(const MOE_EP_LDS char* __restrict__ s, int r0, int ks) {
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    if constexpr (KC) {
      const int row = r0 + i, u = ks * 4 + g;
      return *(const MOE_EP_LDS u32x4*)(s + row * (K * 2) + (u ^ (row & 7)) * 16);
    } else {
      const int k = ks * 32 + g * 8 + (i >> 2);
      const int row = r0 + (i & 3) * 4;
      const MOE_EP_LDS char* p = s + k * (T * 2) + ((row >> 3) ^ (k & 3) * 2) * 16 + (row & 7) * 2;
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_EP_LDS s16x4*)p));
      const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_EP_LDS s16x4*)(p + 8 * T)));
      return u32x4{a[0], a[1], b[0], b[1]};
    }
  }
};

// WP x WQ x WK waves share a tile of TP x TQ.
template <class T_, bool PKC, bool QKC, bool GATED, int TP_, int TQ_, int WP, int WQ, int WK, bool DIRECT>
struct Gemm {
  typedef T_ T;
  static constexpr int TP = TP_, TQ = TQ_;
  static constexpr int kThreads = WP * WQ * WK * 64;
  static constexpr int kK = 64 * WK;                              // k of a tile: 64 for each wave
  static constexpr int FP = TP / WP / 16, FQ = TQ / WQ / 16;      // a wave's fragments
  typedef Side<PKC, GATED, TP, kK, kThreads, DIRECT> SideP;
  typedef Side<QKC, false, TQ, kK, kThreads, DIRECT> SideQ;
  static constexpr int kBuffer = SideP::kBytes + SideQ::kBytes;
  static constexpr int kSums = FP * FQ * 1024;                    // bytes of a wave's sums
  static constexpr int kLds = 2 * kBuffer > (WK - 1) * WP * WQ * kSums ? 2 * kBuffer : (WK - 1) * WP * WQ * kSums;
  typedef f32x4 Acc[FP][FQ];
  static_assert(!GATED || FP % 2 == 0, "a wave holds gate and up of a column");

  static __device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
  // Where a wave's part of the tile starts, and its share of k.
  static __device__ __forceinline__ int wave_p() { return wave() % WP * (TP / WP); }
  static __device__ __forceinline__ int wave_q() { return wave() / WP % WQ * (TQ / WQ); }
  static __device__ __forceinline__ int wave_k() { return wave() / (WP * WQ); }

  typedef u32x4 FragsP[2][FP];
  typedef u32x4 FragsQ[2][FQ];
  // The fragments of 32 k (0 or 1 of the wave's) of the tile at s, into set.
  static __device__ __forceinline__ void frags(const MOE_EP_LDS char* __restrict__ s, FragsP& p, FragsQ& q, int ks) {
#pragma unroll
    for (int j = 0; j < FQ; ++j) q[ks][j] = SideQ::frag(s + SideP::kBytes, wave_q() + j * 16, wave_k() * 2 + ks);
#pragma unroll
    for (int i = 0; i < FP; ++i) p[ks][i] = SideP::frag(s, wave_p() + i * 16, wave_k() * 2 + ks);
  }
  // One set's products, with the reads of the other set between them.
  static __device__ __forceinline__ void products(const FragsP& p, const FragsQ& q, int ks, Acc& acc) {
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
      for (int j = 0; j < FQ; ++j) acc[i][j] = T::mfma(p[ks][i], q[ks][j], acc[i][j]);
    constexpr int kRead = 0x100, kMfma = 0x008;           // sched_group_barrier's classes
    constexpr int reads = SideP::kReads * FP + SideQ::kReads * FQ, count = FP * FQ;
    constexpr int each = (reads + count - 1) / count;
#pragma unroll
    for (int i = 0; i < count; ++i) {
      if (i * each < reads) __builtin_amdgcn_sched_group_barrier(kRead, each, 0);
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    }
  }

  // Every wave's LDS accesses so far, and its loads to LDS, are done.
  static __device__ __forceinline__ void meet() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070);                   // vmcnt(0), lgkmcnt(0); loads to LDS count as memory's
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
  }

  // The same where nothing is loaded to LDS: loads to registers stay under way.
  static __device__ __forceinline__ void meet_lds() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_waitcnt(0xC07F);                   // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    __builtin_amdgcn_sched_barrier(0);
  }

  static __device__ __forceinline__ void load(MOE_EP_LDS char* __restrict__ dst, SideP& sp, SideQ& sq) {
    sp.load(dst);
    sq.load(dst + SideP::kBytes);
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

  // What a wave holds of a tile on its way through registers.
  struct Held {
    u32x4 p[DIRECT ? 1 : SideP::kLoads], q[DIRECT ? 1 : SideQ::kLoads];
  };
  static __device__ __forceinline__ void fetch(Held& h, SideP& sp, SideQ& sq, int left) {
    if constexpr (!DIRECT) {
      if (left > 0) {
        sp.fetch(h.p, left);
        sq.fetch(h.q, left);
      }
    }
  }

  // One tile of k at `cur`, its first 32 k already in the fragments; leaves
  // the first of the tile at `nxt` there.  `left`: of k from the tile after
  // that one on, which goes to `dst`: cur's place, when all waves have read
  // it (through registers, it was fetched a step ago, and the one behind it,
  // with `behind`, is now).  Places of their own for the compiler, which would wait for the
  // loads to LDS before each read otherwise; what orders them is meet().
  static __device__ __forceinline__ void step(const MOE_EP_LDS char* __restrict__ cur,
                                              const MOE_EP_LDS char* __restrict__ nxt, MOE_EP_LDS char* __restrict__ dst,
                                              SideP& sp, SideQ& sq, FragsP& p, FragsQ& q, Acc& acc, Held& held,
                                              int left, int behind) {
    frags(cur, p, q, 1);
    products(p, q, 0, acc);
    if constexpr (DIRECT) {
      meet();
      if (left >= kK) load(dst, sp, sq);
      else if (left > 0) fill(dst, sp, sq, left);
    } else {
      meet_lds();
      if (left > 0) {
        SideP::put(dst, held.p);
        SideQ::put(dst + SideP::kBytes, held.q);
        fetch(held, sp, sq, behind);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    frags(nxt, p, q, 0);
    products(p, q, 1, acc);
    __builtin_amdgcn_sched_barrier(0);
  }

  static __device__ __forceinline__ void clear(Acc& acc) {
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
      for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  }

  // Sends out the first two tiles of k.
  static __device__ __forceinline__ void begin(MOE_EP_LDS char* lds, SideP& sp, SideQ& sq, int K) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int left = K - b * kK;
      if (DIRECT && left >= kK) load(lds + b * kBuffer, sp, sq);
      else if (left > 0) fill(lds + b * kBuffer, sp, sq, left);
    }
  }
  // After begin(): adds the wave's products over its share of K to acc.
  static __device__ __forceinline__ void loop(MOE_EP_LDS char* lds, SideP& sp, SideQ& sq, int K, Acc& acc) {
    if (K <= 0) return;
    Held held;
    fetch(held, sp, sq, K - 2 * kK);
    meet();
    FragsP p;
    FragsQ q;
    frags(lds, p, q, 0);
    int cur = 0;
#pragma unroll 1
    for (int left = K; left > 0; left -= kK) {
      // (past the last tile nxt is read for nothing, inside lds)
      step(lds + cur, lds + (kBuffer - cur), lds + cur, sp, sq, p, q, acc, held, left - 2 * kK,
           left - 3 * kK);
      cur = kBuffer - cur;
    }
  }
  // begin() and loop() over the same K (at least 1) twice: back(count) is called
  // when the last of the first time's `count` tiles has been sent for, between()
  // when its products are made.
  template <class Back, class Between>
  static __device__ __forceinline__ void loop_twice(MOE_EP_LDS char* lds, SideP& sp, SideQ& sq, int K, Acc& acc,
                                                    const Back& back, const Between& between) {
    const int count = (K + kK - 1) / kK;
    auto left = [&](int t) { return t < 2 * count ? K - (t < count ? t : t - count) * kK : 0; };
    auto sent = [&](int t) {
      if (t == count - 1) back(count);
    };
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (DIRECT && left(b) >= kK) load(lds + b * kBuffer, sp, sq);
      else fill(lds + b * kBuffer, sp, sq, left(b));
      sent(b);
    }
    Held held;
    fetch(held, sp, sq, left(2));
    if (!DIRECT) sent(2);
    meet();
    FragsP p;
    FragsQ q;
    frags(lds, p, q, 0);
    int cur = 0;
#pragma unroll 1
    for (int t = 0; t < 2 * count; ++t) {
      step(lds + cur, lds + (kBuffer - cur), lds + cur, sp, sq, p, q, acc, held, left(t + 2), left(t + 3));
      sent(t + (DIRECT ? 2 : 3));
      if (t == count - 1) between();
      cur = kBuffer - cur;
    }
  }
  // Adds the sums of the waves that share k.  They are in the waves with
  // wave_k() 0; the others return false.
  static __device__ __forceinline__ bool join(MOE_EP_LDS char* lds, Acc& acc) {
    if constexpr (WK > 1) {
      meet();
      const int lane = threadIdx.x & 63, w = wave() % (WP * WQ);
      MOE_EP_LDS f32x4* sums = (MOE_EP_LDS f32x4*)lds;
      if (wave_k() > 0) {
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
          for (int j = 0; j < FQ; ++j)
            sums[(((wave_k() - 1) * WP * WQ + w) * (FP * FQ) + i * FQ + j) * 64 + lane] = acc[i][j];
      }
      __syncthreads();
      if (wave_k() > 0) return false;
#pragma unroll
      for (int o = 0; o < WK - 1; ++o)
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
          for (int j = 0; j < FQ; ++j) acc[i][j] += sums[((o * WP * WQ + w) * (FP * FQ) + i * FQ + j) * 64 + lane];
    }
    return true;
  }
};

// Which tile a workgroup makes.  Each XCD (workgroups go to the 8 of them in
// turn) takes a run of tiles, and a run goes through 4 tiles of q before the
// next p, so that what an XCD reads at one time stays in its L2 (8192 x 4096 x
// 7168 in a trial of this loop: 413 us with 1, 405 with 4, 414 with 8, 437 with 32).
__device__ __forceinline__ void tile_of(int ptiles, int qtiles, int* pt, int* qt) {
  const int n = gridDim.x, x = blockIdx.x % 8, i = blockIdx.x / 8, per = n / 8, rem = n % 8;
  const int b = x * per + min(x, rem) + i;
  constexpr int kGroup = 4;
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
