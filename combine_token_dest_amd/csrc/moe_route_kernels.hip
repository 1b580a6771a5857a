// gfx950 kernel of the router's selection (moe_ep_route).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "moe_experts_internal.h"
#include "moe_route_device.h"

namespace moe_ep_detail {
namespace {

constexpr int kRouteThreads = 256;

// One token of 256 experts in groups 6.2 us, 1024 tokens of 256 experts 5.1, 8192
// of 128 with weights by the softmax over all (16 lanes to a token) 7.4, of which
// the denominator in float64 takes 0.9 more than in float32; in float32 and with a
// wave to a token the last took 11.7.
template <typename V, int LPT, int VPL, bool GROUPS>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteKArgs a) {
  constexpr int kTokens = 64 / LPT;
  extern __shared__ double choices[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane & (LPT - 1);
  const int64_t token = ((int64_t)blockIdx.x * (kRouteThreads / 64) + wave) * kTokens + lane / LPT;
  int id;
  float weight;
  route_token<V, LPT, VPL, GROUPS>(a, token < a.n ? token : a.n - 1, choices + wave * a.num_experts, &id, &weight);
  if (token < a.n && sub < a.top_k) {
    a.ids[token * a.top_k + sub] = id;
    a.weights[token * a.top_k + sub] = weight;
  }
}

template <typename V, int LPT, bool GROUPS>
void start_route(const RouteKArgs& a, hipStream_t stream) {
  constexpr int kPerBlock = kRouteThreads / 64 * (64 / LPT);
  const int grid = (int)(((int64_t)a.n + kPerBlock - 1) / kPerBlock);
  const size_t lds = GROUPS ? (size_t)(kRouteThreads / 64) * a.num_experts * sizeof(double) : 0;
  const int vpl = (a.num_experts + LPT - 1) / LPT;
  if (vpl <= 1) route_kernel<V, LPT, 1, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
  else if (vpl <= 2) route_kernel<V, LPT, 2, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
  else if (vpl <= 4) route_kernel<V, LPT, 4, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
  else if (vpl <= 8) route_kernel<V, LPT, 8, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
  else route_kernel<V, LPT, 16, GROUPS><<<grid, kRouteThreads, lds, stream>>>(a);
}

}  // namespace

hipError_t launch_route(const RouteKArgs& all, hipStream_t stream) {
  // A launch has fewer than 2^32 threads in x, and a token up to 64.
  constexpr int kMost = 1 << 24;
  RouteKArgs a = all;
  for (int64_t t = 0; t < all.n; t += kMost) {
    a.n = (int32_t)std::min<int64_t>(kMost, all.n - t);
    a.logits = static_cast<const uint8_t*>(all.logits) + t * all.logits_stride * (all.logits_dtype == MOE_EP_F32 ? 4 : 2);
    a.ids = all.ids + t * all.top_k;
    a.weights = all.weights + t * all.top_k;
    if (a.num_groups > 1) start_route<double, 64, true>(a, stream);
    else if (a.bias) start_route<double, 64, false>(a, stream);
    else if (a.n >= 2048 && a.num_experts <= 256 && a.top_k <= 16) start_route<float, 16, false>(a, stream);
    else start_route<float, 64, false>(a, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe_ep_detail
