// Internal interface between the host code of the expert-side operators
// (moe_experts_api.cpp) and their gfx950 kernels (moe_experts_kernels.hip):
// the router's selection, the experts' linear product and the whole layer.
// Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "moe_ep.h"

namespace moe_ep_detail {

// Records a failed call's message for moe_ep_last_error() and returns status
// (moe_ep_api.cpp).
int report(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Tokens of one pass over the experts' weights: a workgroup keeps an
// expert's list of tokens in LDS (8 KiB).  Longer calls run several passes.
constexpr int kPassTokens = 2048;
// Tokens whose output tile one workgroup of the down product sums in LDS:
// 64 bytes a token and wave, 64 KiB at eight waves.
constexpr int kChunkTokens = 128;
constexpr int kMaxChunks = kPassTokens / kChunkTokens;
// Waves of a workgroup of the expert kernels; they share the sum over k.
constexpr int kExpertWaves = 8;

// The activations between the layer's products are float32 values, whole:
// bfloat16 parts of 8 bits each are what the down product's matrix
// instructions take.  (Two parts of the activations' own type would halve
// these instructions' cost, but keep 16 bits for bfloat16, and float16 keeps
// nothing of small values and ends at 131008.)
constexpr int kParts = 3;

// Waves of a workgroup of the kernels for many tokens to an expert.
constexpr int kWideWaves = 4;

struct RouteKArgs {
  const void* logits;
  int64_t logits_stride;      // elements
  const float* bias;          // [num_experts] or NULL
  int32_t* ids;               // [n, top_k]
  float* weights;             // [n, top_k]
  int32_t n;
  int32_t num_experts;
  int32_t top_k;
  int32_t logits_dtype;
  int32_t score;
  int32_t num_groups;
  int32_t top_groups;
  int32_t group_top;
  int32_t renormalize;
  int32_t invalid_id;
  float scale;
};

// One expert matrix [N, K] per expert.
struct WeightK {
  const uint8_t* data;
  const uint16_t* scales;     // 4-bit weights only
  int64_t expert_bytes;       // of data, per expert
  int64_t expert_scales;      // scale elements per expert
  int32_t rows;               // N
  int32_t cols;               // K
  int32_t kblocks;            // 4-bit: tiles of 128 columns per row
  int32_t groups;             // 4-bit: scale groups per row (kblocks * 128 / group size)
};

// What the layer's first kernel leaves in the workspace for its second.
// Slot a is one expert that may have tokens (a pair's or an expert's index).
struct PlanK {
  int32_t* head;              // [chunks, slots]: pack_head() of the slot's tokens in the chunk
  void* pair;                 // [slots, n] of {token << 6 | top-k slot, weight}, tokens ascending
  // The activations: their parts, bfloat16 [kParts, n * top_k, act_stride]; for
  // down_kernel with dense weights float32 [n * top_k, act_stride].
  void* act;
  int64_t act_plane;          // elements from a part to the next; 0: float32
  int32_t act_stride;
  int32_t slots;
};

// A slot's tokens in one chunk: how many (up to 128), where they start in
// its list (below 2048), and its expert (below 1024).
#ifdef __HIP__
#define MOE_EP_HD __host__ __device__ __forceinline__
#else
#define MOE_EP_HD inline
#endif
static_assert(kChunkTokens <= 255 && kPassTokens <= 2048 && MOE_EP_MAX_EXPERTS <= 1024, "fields of a packed head");
MOE_EP_HD int32_t pack_head(int count, int start, int expert) {
  return (int32_t)((uint32_t)count | (uint32_t)(count ? start : 0) << 8 | (uint32_t)expert << 19);
}
MOE_EP_HD int head_count(int32_t h) { return h & 255; }
MOE_EP_HD int head_start(int32_t h) { return (h >> 8) & 2047; }
MOE_EP_HD int head_expert(int32_t h) { return (h >> 19) & 1023; }

// The product whose rows are gathered by expert: expert_linear, and the
// layer's gate and up product.
struct RowsKArgs {
  const uint16_t* x;
  int64_t x_stride;
  const int32_t* ids;         // [n, top_k], or NULL: every row is expert 0's
  const float* topk_weights;  // [n, top_k] or NULL (layer only)
  WeightK w;
  PlanK plan;                 // layer only
  void* out;                  // linear only
  int64_t out_stride;
  int32_t out_f32;
  int32_t n;
  int32_t top_k;
  int32_t offset;             // first expert id
  int32_t num_experts;
  int32_t by_pair;            // slots are (token, k) pairs, else experts
  int32_t inter;              // gate and up: intermediate size; else the rows of w
  int32_t wide;               // many tokens to an expert (wide_kernel)
  float* pair_out;            // wide down product: [n * top_k, pair_stride], each pair's weighted product
  int64_t pair_stride;
  int32_t split;              // waves that share a tile (set by the launcher)
  int32_t tiles_per_block;    // (set by the launcher)
  int32_t busiest_first;      // wide: blockIdx.y counts the experts by their pairs (set by the launcher)
};

// The same for a few tokens that the kernel routes itself.
struct RowsRoutedKArgs : RowsKArgs {
  RouteKArgs route;
};
// The most such tokens (a wave of a workgroup for each), pairs and experts.
constexpr int kRoutedTokens = kExpertWaves, kFewPairs = 64, kRoutedExperts = 256;

// The layer's down product, summed over the experts of each token.
struct DownKArgs {
  WeightK w;
  PlanK plan;
  void* out;
  int64_t out_stride;
  int32_t out_f32;
  int32_t n;
  int32_t top_k;
  int32_t tiles;              // of 16 output columns
  int32_t chunks;
};

hipError_t launch_route(const RouteKArgs& a, hipStream_t stream);
// dtype: MOE_EP_BF16 or MOE_EP_F16; group: 0 for dense weights, else 32, 64 or 128.
hipError_t launch_expert_linear(const RowsKArgs& a, int dtype, int group, hipStream_t stream);
hipError_t launch_gate_up(const RowsKArgs& a, int dtype, int group, hipStream_t stream);
hipError_t launch_gate_up_routed(const RowsRoutedKArgs& a, int dtype, int group, hipStream_t stream);
hipError_t launch_down(const DownKArgs& a, int dtype, int group, hipStream_t stream);
// The down product for many tokens to an expert, and the sum over each token's pairs.
hipError_t launch_wide_down(const RowsKArgs& a, int dtype, int group, hipStream_t stream);

}  // namespace moe_ep_detail
