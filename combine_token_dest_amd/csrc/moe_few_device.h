// Products of a matrix's rows with a few rows of x (up to 16 NT), for the
// dense operators at decode sizes.
//
// What such a call cannot do without is one read of the weights, so it is
// bound by streaming them from HBM: one row of 4096 x 7168 gated takes 10.7 us,
// 5.5 TB/s.  A workgroup takes 16 rows of the matrix,
// the A operand of v_mfma_f32_16x16x32, and rows of x are the columns of B;
// its waves share k, 64 k (128 bytes of a row) a step in turn, each with
// kDepth steps' loads under way, and their sums are added through LDS in a
// fixed order.
//
// As operands, 16 lanes side by side hold 16 rows; loaded like that, each
// would touch a cache line of its own, and the first cache's look-ups would
// be the limit.  So 8 lanes load a row's 128 bytes, and at its use a step goes
// through the wave's own piece of LDS, which hands it out as operands: unit u
// of row r is at u ^ (r & 7) there.
//
// Workgroups begin at different k and go around, so that rows that start in
// the same channel of L2 are not all asked for at once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_gemm_device.h"

namespace moe_ep_detail {
namespace {

// The sums of MT x 16 rows of A and NT x 16 rows of x over this wave's steps
// of 64 k: acc[m][t], in a lane rows 4 (lane / 16) + e of A, row lane & 15 of
// x.
template <class T, int MT, int NT, int WAVES>
struct Few {
  static constexpr int kSets = MT + NT;
  static constexpr int kMost = (WAVES > 8 ? 72 : 104) / (8 * kSets);    // 16 waves have 128 registers each
  static constexpr int kDepth = kMost > 4 ? 4 : kMost;
  static constexpr int kLds = kSets * 2048;               // bytes of a wave's piece
  static_assert(kDepth >= 2, "a step's loads go out while another's are used");
  struct Stage {
    u32x4 v[kSets][2];
  };

  const uint16_t* p[kSets][2];   // the lane's unit of rows lane / 8 and 8 + lane / 8, in step 0
  int steps;                  // whole steps of 64 k that the waves share
  int turn;                   // step 0's place among them
  MOE_EP_LDS char* lds;

  static __device__ __forceinline__ int lane() { return threadIdx.x & 63; }
  static __device__ __forceinline__ int unit() { return (lane() & 7) ^ (lane() >> 3); }

  // a(m, i) and b(t, i) are row i of each set; the steps begin at step `first`
  // of the rows; `piece` is the wave's LDS.
  template <class A, class B>
  __device__ __forceinline__ void aim(A a, B b, int64_t first, int count, int workgroup, void* piece) {
    lds = (MOE_EP_LDS char*)piece;
#pragma unroll
    for (int s = 0; s < kSets; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = h * 8 + (lane() >> 3);
        p[s][h] = (s < MT ? a(s, row) : b(s - MT, row)) + first * 64 + unit() * 8;
      }
    steps = count;
    // 19 steps are 2432 bytes: neighbours are in channels of their own
    turn = count > 0 ? workgroup * 19 % count : 0;
  }

  __device__ __forceinline__ void load(Stage& st, int step) const {
    const int place = step + turn, at = (place >= steps ? place - steps : place) * 64;
#pragma unroll
    for (int s = 0; s < kSets; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) st.v[s][h] = load_any8(p[s][h] + at);
  }
  // The step after the whole ones, of which only `left` (1..63) k exist.
  __device__ __forceinline__ void load_cut(Stage& st, int left) const {
    const int at = steps * 64, have = left - unit() * 8;
#pragma unroll
    for (int s = 0; s < kSets; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) st.v[s][h] = load_any8(p[s][h] + at + (min(have, 8) - 8));
#pragma unroll
    for (int s = 0; s < kSets; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) st.v[s][h] = keep_last(st.v[s][h], have);
  }
  // (A wave's LDS accesses take their turn, so the next step's writes come
  // after this one's reads.)
  __device__ __forceinline__ void add(const Stage& st, f32x4 (&acc)[MT][NT]) const {
#pragma unroll
    for (int s = 0; s < kSets; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) *(MOE_EP_LDS u32x4*)(lds + s * 2048 + h * 1024 + lane() * 16) = st.v[s][h];
    const int row = lane() & 15;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4 f[kSets];
#pragma unroll
      for (int s = 0; s < kSets; ++s)
        f[s] = *(const MOE_EP_LDS u32x4*)(lds + s * 2048 + row * 128 + ((ks * 4 + (lane() >> 4)) ^ (row & 7)) * 16);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = T::mfma(f[m], f[MT + t], acc[m][t]);
    }
  }

  Stage stage[kDepth];
  // Sends out the first loads of steps first, first + stride, ...
  __device__ __forceinline__ void prime(int first, int stride) {
    if (first >= steps) return;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(stage[d], min(first + d * stride, steps - 1));
  }
  // Goes through the steps, kDepth at a time.  No branch stands between a load
  // and its use (where paths join, the wait for a load becomes a wait for
  // all): past the last step the loads repeat it.
  __device__ __forceinline__ void run(int first, int stride, f32x4 (&acc)[MT][NT]) {
    if (first >= steps) return;
    int s = first;
    for (; s + kDepth * stride < steps; s += kDepth * stride) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        add(stage[d], acc);
        load(stage[d], min(s + (d + kDepth) * stride, steps - 1));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (s + d * stride < steps) add(stage[d], acc);
  }
  __device__ __forceinline__ void tail(int left, f32x4 (&acc)[MT][NT]) {
    Stage st;
    load_cut(st, left);
    add(st, acc);
  }
};

}  // namespace
}  // namespace moe_ep_detail
