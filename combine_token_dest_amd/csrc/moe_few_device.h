// Products of a matrix's rows with a few rows of x (up to 16 NT), for the
// dense operators at decode sizes.
//
// What such a call cannot do without is one read of the weights, so it is
// bound by streaming them from HBM.  A workgroup takes 16 rows of the matrix,
// the A operand of v_mfma_f32_16x16x32, and rows of x are the columns of B;
// its waves share k, 64 k (128 bytes of a row) a step in turn, each with
// kDepth steps' loads under way, and their sums are added through LDS in a
// fixed order.  Nothing goes through LDS on the way in: a weight is used by
// one wave only, and x comes from L2.
//
// Workgroups begin at different k and go around: rows of 4096 elements start
// in the same channel of L2, and all workgroups at one k would ask the same
// few channels.
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
  static constexpr int kRegs = 8 * (MT + NT);             // of a step
  static constexpr int kMost = (WAVES > 8 ? 72 : 104) / kRegs;    // 16 waves have 128 registers each
  static constexpr int kDepth = kMost > 4 ? 4 : kMost;
  static_assert(kDepth >= 2, "a step's loads go out while another's are used");
  struct Stage {
    u32x4 a[MT][2], b[NT][2];
  };

  const uint16_t* a[MT];      // the lane's rows, at its first k of a step
  const uint16_t* b[NT];

  int steps;                  // whole steps of 64 k that the waves share
  int turn;                   // step 0's place among them

  // The rows of the lane (lane & 15), their steps' number, and who begins where.
  __device__ __forceinline__ void aim(const uint16_t* const (&ra)[MT], const uint16_t* const (&rb)[NT], int64_t first,
                                      int count, int workgroup) {
    const int64_t k = first * 64 + (threadIdx.x & 63) / 16 * 8;
    steps = count;
    // 19 steps are 2432 bytes: neighbours are in channels of their own
    turn = count > 0 ? workgroup * 19 % count : 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) a[m] = ra[m] + k;
#pragma unroll
    for (int t = 0; t < NT; ++t) b[t] = rb[t] + k;
  }

  __device__ __forceinline__ void load(Stage& s, int step) const {
    const int place = step + turn, at = (place >= steps ? place - steps : place) * 64;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int m = 0; m < MT; ++m) s.a[m][h] = load_any8(a[m] + at + h * 32);
#pragma unroll
      for (int t = 0; t < NT; ++t) s.b[t][h] = load_any8(b[t] + at + h * 32);
    }
  }
  // The step after the whole ones, of which only `left` (1..63) k exist.
  __device__ __forceinline__ void load_cut(Stage& s, int left) const {
    const int at = steps * 64;
    const int k = (threadIdx.x & 63) / 16 * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int have = left - k - h * 32;
#pragma unroll
      for (int i = 0; i < MT + NT; ++i) {
        const uint16_t* p = (i < MT ? a[i < MT ? i : 0] : b[i < MT ? 0 : i - MT]) + at + h * 32;
        u32x4 v = {0, 0, 0, 0};
        if (have >= 8) v = load_any8(p);
        else if (have > 0) v = keep_last(load_any8(p + (have - 8)), have);
        if (i < MT) s.a[i < MT ? i : 0][h] = v;
        else s.b[i < MT ? 0 : i - MT][h] = v;
      }
    }
  }
  static __device__ __forceinline__ void add(const Stage& s, f32x4 (&acc)[MT][NT]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = T::mfma(s.a[m][h], s.b[t][h], acc[m][t]);
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
    Stage s;
    load_cut(s, left);
    add(s, acc);
  }
};

}  // namespace
}  // namespace moe_ep_detail
