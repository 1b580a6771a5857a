// gfx950 kernel of a shared projection with low-rank adapters:
//   y[r] = W x[r] + s_a B_a (A_a x[r]), a = ids[r],
// where low[r] = A_a x[r] (float32) has been made by expert_linear's kernels.
//
// The shared product is that of moe_gemm_device.h.  Behind it, while the sums
// are still in registers, a wave goes through the adapters that its rows name,
// one after another: B_a's rows times the low-rank values by matrix
// instructions, added to the rows that have this adapter and to no others (a
// row's result never meets another adapter's B, whatever is in it).  The low
// values go in as three bfloat16 each, float32's 24 bits.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dense_internal.h"
#include "moe_gemm_device.h"

namespace moe_ep_detail {
namespace {

// Eight elements of a row of `rank` from k on; zeros past it.
__device__ __forceinline__ u32x4 b_elements(const uint16_t* row, int k, int rank) {
  if (k + 8 <= rank) return load_any8(row + k);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (k + e < rank) v[e >> 1] |= (uint32_t)row[k + e] << (e & 1) * 16;
  return v;
}

// Eight low values times the scale, in parts.
__device__ __forceinline__ void low_parts(const float* row, int k, int rank, float scale, u32x4 (&part)[kParts]) {
  u32x4 v[2];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = k + e < rank ? __float_as_uint(row[k + e] * scale) : 0u;
  split_floats(v, part);
}

template <class G>
__global__ void __launch_bounds__(G::kThreads, G::kThreads / 256) adapter_kernel(AdapterKArgs a) {
  typedef typename G::T T;
  __shared__ __attribute__((aligned(1024))) char lds[G::kLds];
  int pt, qt;
  tile_of(a.ptiles, a.qtiles, &pt, &qt);
  typename G::SideP sp;
  typename G::SideQ sq;
  sp.aim(a.w, pt * G::TP);
  sq.aim(a.x, qt * G::TQ);
  typename G::Acc acc;
  if (!G::run((MOE_EP_LDS char*)lds, sp, sq, a.k, acc)) return;

  const int lane = threadIdx.x & 63, quarter = lane >> 4;
  const int N = a.w.rows, R = a.rank;
#pragma unroll
  for (int j = 0; j < G::FQ; ++j) {
    const int q = qt * G::TQ + G::wave_q() + j * 16 + (lane & 15);
    const bool here = q < a.x.rows;
    int id = here ? a.ids[q] : -1;
    if (id < 0 || id >= a.adapters) id = -1;
    uint64_t pending = __ballot(id >= 0);
    while (pending) {
      const int ad = __builtin_amdgcn_readlane(id, __builtin_ctzll(pending));
      pending &= ~__ballot(id == ad);
      const float scale = a.scales ? a.scales[ad] : 1.0f;
      const float* low = a.low + (int64_t)(here ? q : 0) * R;
#pragma unroll
      for (int i = 0; i < G::FP; ++i) {
        const int p = min(pt * G::TP + G::wave_p() + i * 16 + (lane & 15), N - 1);
        const uint16_t* b = a.b + ((int64_t)ad * N + p) * R;
        f32x4 sum = {0, 0, 0, 0};
        for (int k = 0; k < R; k += 32) {
          u32x4 part[kParts];
          low_parts(low, k + quarter * 8, R, scale, part);
          u32x4 v[2] = {b_elements(b, k + quarter * 8, R), {}};
          if constexpr (std::is_same<T, F16>::value) {
            const u32x4 w = v[0];
            split_f16(w, &v[0], &v[1]);
          }
#pragma unroll
          for (int pl = 0; pl < kParts; ++pl) {
            sum = BF16::mfma(v[0], part[pl], sum);
            if constexpr (std::is_same<T, F16>::value) sum = BF16::mfma(v[1], part[pl], sum);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = id == ad ? acc[i][j][e] + sum[e] : acc[i][j][e];
      }
    }
    if (!here) continue;
#pragma unroll
    for (int i = 0; i < G::FP; ++i) {
      const int c = pt * G::TP + G::wave_p() + i * 16 + quarter * 4;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e];
      store4<T>(a.out, q * a.out_stride + c, a.out_f32, N - c, v);
    }
  }
}

template <class G>
hipError_t adapter_tiles(AdapterKArgs a, hipStream_t stream) {
  a.ptiles = tiles(a.w.rows, G::TP);
  a.qtiles = tiles(a.x.rows, G::TQ);
  adapter_kernel<G><<<dim3(a.ptiles * a.qtiles), dim3(G::kThreads), 0, stream>>>(a);
  return hipGetLastError();
}
template <class T>
hipError_t adapter(const AdapterKArgs& a, hipStream_t stream) {
  const bool direct = a.w.whole && a.x.whole;
  switch (tile_size(a.w.rows, a.x.rows, direct)) {
    case 256: return adapter_tiles<Gemm<T, true, true, false, 256, 256, 2, 4, 1, true>>(a, stream);
    case 128:
      return direct ? adapter_tiles<Gemm<T, true, true, false, 128, 128, 2, 2, 2, true>>(a, stream)
                    : adapter_tiles<Gemm<T, true, true, false, 128, 128, 2, 2, 2, false>>(a, stream);
    default:
      return direct ? adapter_tiles<Gemm<T, true, true, false, 64, 64, 2, 2, 4, true>>(a, stream)
                    : adapter_tiles<Gemm<T, true, true, false, 64, 64, 2, 2, 4, false>>(a, stream);
  }
}

}  // namespace

hipError_t launch_adapter(const AdapterKArgs& a, int dtype, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? adapter<BF16>(a, stream) : adapter<F16>(a, stream);
}

}  // namespace moe_ep_detail
