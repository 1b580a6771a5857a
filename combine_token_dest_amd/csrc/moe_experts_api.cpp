// C-ABI host side of the expert-side operators: argument checks, the layer's
// workspace layout, passes of at most kPassTokens tokens, and launches.
// Every check comes before the first launch, so a refused call leaves no
// device work behind.

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "moe_args_internal.h"
#include "moe_ep.h"
#include "moe_experts_internal.h"

using namespace moe_ep_detail;

namespace {

int check_router(const moe_ep_router& r) {
  if (r.num_experts < 1 || r.num_experts > MOE_EP_MAX_EXPERTS)
    return report(MOE_EP_ERR_INVALID_ARG, "router num_experts %d outside [1, %d]", r.num_experts, MOE_EP_MAX_EXPERTS);
  if (r.top_k < 1 || r.top_k > MOE_EP_MAX_TOPK || r.top_k > r.num_experts)
    return report(MOE_EP_ERR_INVALID_ARG, "router top_k %d outside [1, min(%d, %d experts)]", r.top_k, MOE_EP_MAX_TOPK,
                  r.num_experts);
  if (r.score != MOE_EP_SCORE_SOFTMAX && r.score != MOE_EP_SCORE_SIGMOID)
    return report(MOE_EP_ERR_INVALID_ARG, "router score %d unknown", r.score);
  if (r.num_groups < 1 || r.num_groups > MOE_EP_MAX_GROUPS || r.num_experts % r.num_groups != 0)
    return report(MOE_EP_ERR_INVALID_ARG, "num_groups %d is above %d or does not divide %d experts", r.num_groups,
                  MOE_EP_MAX_GROUPS, r.num_experts);
  if (r.top_groups < 1 || r.top_groups > r.num_groups)
    return report(MOE_EP_ERR_INVALID_ARG, "top_groups %d outside [1, %d]", r.top_groups, r.num_groups);
  if (r.top_groups * (r.num_experts / r.num_groups) < r.top_k)
    return report(MOE_EP_ERR_INVALID_ARG, "%d groups of %d experts hold fewer than top_k %d", r.top_groups,
                  r.num_experts / r.num_groups, r.top_k);
  if (r.group_top != 1 && r.group_top != 2)
    return report(MOE_EP_ERR_INVALID_ARG, "group_top %d is not 1 or 2", r.group_top);
  if (!aligned_to(r.bias, 4)) return report(MOE_EP_ERR_ALIGN, "router bias not 4-byte aligned");
  return MOE_EP_OK;
}

int check_logits(const moe_ep_router& r, const void* logits, int dtype, int64_t stride, int n) {
  const int esz = elem_bytes(dtype);
  if (esz == 0) return report(MOE_EP_ERR_INVALID_ARG, "unknown logits dtype %d", dtype);
  if (stride < 0 || (n > 1 && stride != 0 && stride < r.num_experts) || stride > INT64_MAX / 8 / std::max(n, 1))
    return report(MOE_EP_ERR_INVALID_ARG, "logits stride %lld with %d experts", (long long)stride, r.num_experts);
  if (n > 0 && !logits) return report(MOE_EP_ERR_INVALID_ARG, "NULL logits with %d tokens", n);
  if (!aligned_to(logits, esz)) return report(MOE_EP_ERR_ALIGN, "logits not aligned to their element");
  return MOE_EP_OK;
}

RouteKArgs route_args(const moe_ep_router& r, const void* logits, int dtype, int64_t stride, int n, int32_t* ids,
                      float* weights) {
  RouteKArgs k;
  k.logits = logits;
  k.logits_stride = stride;
  k.bias = r.bias;
  k.ids = ids;
  k.weights = weights;
  k.n = n;
  k.num_experts = r.num_experts;
  k.top_k = r.top_k;
  k.logits_dtype = dtype;
  k.score = r.score;
  k.num_groups = r.num_groups;
  k.top_groups = r.top_groups;
  k.group_top = r.group_top;
  k.renormalize = r.renormalize;
  k.invalid_id = r.invalid_expert_id;
  k.scale = r.scale;
  return k;
}

// Checks one weight set [experts, N, K] and fills the kernels' view of it.
int make_weight(const moe_ep_weight& w, int64_t N, int64_t K, const char* what, WeightK* k) {
  const int g = w.group_size;
  if (g != 0 && g != 32 && g != 64 && g != 128)
    return report(MOE_EP_ERR_INVALID_ARG, "%s: group_size %d is not 0, 32, 64 or 128", what, g);
  if (!w.data) return report(MOE_EP_ERR_INVALID_ARG, "%s: NULL weight data", what);
  k->data = static_cast<const uint8_t*>(w.data);
  k->scales = static_cast<const uint16_t*>(w.scales);
  k->rows = (int32_t)N;
  k->cols = (int32_t)K;
  k->kblocks = (int32_t)((K + 127) / 128);
  k->groups = g ? k->kblocks * (128 / g) : 0;
  if (g == 0) {
    if (!aligned_to(w.data, 2)) return report(MOE_EP_ERR_ALIGN, "%s: weights not 2-byte aligned", what);
    k->expert_bytes = N * K * 2;
    k->expert_scales = 0;
  } else {
    if (!w.scales) return report(MOE_EP_ERR_INVALID_ARG, "%s: NULL scales with group_size %d", what, g);
    if (!aligned_to(w.data, 16) || !aligned_to(w.scales, 16))
      return report(MOE_EP_ERR_ALIGN, "%s: 4-bit weights and scales must be 16-byte aligned", what);
    k->expert_bytes = (N + 15) / 16 * k->kblocks * 1024;
    k->expert_scales = (N + 15) / 16 * k->groups * 16;
  }
  return MOE_EP_OK;
}

int check_experts(int num_experts, int offset) {
  if (num_experts < 1 || num_experts > MOE_EP_MAX_EXPERTS)
    return report(MOE_EP_ERR_INVALID_ARG, "num_experts %d outside [1, %d]", num_experts, MOE_EP_MAX_EXPERTS);
  if (offset < 0 || offset > INT32_MAX - num_experts)
    return report(MOE_EP_ERR_INVALID_ARG, "expert_offset %d with %d experts", offset, num_experts);
  return MOE_EP_OK;
}

// Whether the kernels for many tokens to an expert take a pass of n tokens
// with top_k experts each (moe_experts_kernels.hip, wide_kernel).  The narrow
// ones take four (4-bit) or eight (dense) tokens at a time and read the
// weights again for each such pass, from L2 at best, but share a row's sum
// over k between waves; the wide ones read the weights once per 48 tokens, but
// a workgroup covers `tile_rows` of the weights' rows and goes through all of
// k alone.  Measured, narrow / wide in us:
//   layer, 64 experts, top-8, 4096 x 1024, 4 bits: 8 tokens 79 / 79, 16: 113 / 102, 32: 153 / 111, 128: 413 / 132
//   the same dense:                                32 tokens 284 / 302, 64: 390 / 308, 128: 625 / 318
//   one 4-bit matrix 4096 x 4096: 24 rows 15 / 20, 48: 27 / 27, 96: 50 / 27;  4096 x 1024: 12 rows 7.3 / 6.0
//   one dense matrix 4096 x 4096: 48 rows 33 / 35, 96: 63 / 35;  4096 x 1024: 12 rows 7.6 / 11, 48: 17 / 11
// (The experts' tokens are counted as if all of them were chosen here.)
bool is_wide(int64_t n, int top_k, int64_t num_experts, int64_t rows, int tile_rows, int64_t cols, int group) {
  const int64_t pairs = n * top_k;
  const int64_t blocks = (rows + tile_rows - 1) / tile_rows * std::min(pairs, num_experts);
  if (pairs >= num_experts * (group ? 2 : 6) && blocks >= 128) return true;
  const int64_t at_once = num_experts * (group ? 4 : 8), passes = (pairs + at_once - 1) / at_once;
  const int64_t steps = group ? (cols + 127) / 128 : (cols + 63) / 64;
  return passes > (group ? 1 : 2) && passes * blocks >= steps * (group ? 12 : 4);
}

// Workspace of one pass: [ids][weights] with a router, the plan, the
// activations.  Every part starts on 256 bytes.
struct LayerSpace {
  int64_t ids, weights, head, pair, act, pair_out, pair_stride, total;
  int32_t n, slots, act_stride;
  bool wide;
};

int make_space(const moe_ep_layer_args* a, LayerSpace* s) {
  int st = check_experts(a->num_experts, a->expert_offset);
  if (st != MOE_EP_OK) return st;
  if (a->num_tokens < 0) return report(MOE_EP_ERR_INVALID_ARG, "num_tokens %d < 0", a->num_tokens);
  if (a->top_k < 1 || a->top_k > MOE_EP_MAX_TOPK)
    return report(MOE_EP_ERR_INVALID_ARG, "top_k %d outside [1, %d]", a->top_k, MOE_EP_MAX_TOPK);
  if (a->hidden_size < kMinRow || a->hidden_size > kMaxSide)
    return report(MOE_EP_ERR_INVALID_ARG, "hidden_size %d outside [%d, %d]", a->hidden_size, kMinRow, kMaxSide);
  if (a->intermediate_size < kMinRow || a->intermediate_size > kMaxSide)
    return report(MOE_EP_ERR_INVALID_ARG, "intermediate_size %d outside [%d, %d]", a->intermediate_size, kMinRow,
                  kMaxSide);
  s->n = std::min(a->num_tokens, kPassTokens);
  const int64_t pairs = (int64_t)s->n * a->top_k;
  s->slots = (int32_t)std::min<int64_t>(pairs, a->num_experts);
  s->act_stride = (int32_t)up(a->intermediate_size, 16);
  int64_t off = 0;
  auto take = [&off](int64_t bytes) {
    const int64_t at = off;
    off += up(bytes, 256);
    return at;
  };
  s->ids = take(a->router ? pairs * 4 : 0);
  s->weights = take(a->router ? pairs * 4 : 0);
  s->head = take((int64_t)s->slots * kMaxChunks * 4);
  s->pair = take((int64_t)s->slots * s->n * 8);
  s->wide = is_wide(s->n, a->top_k, a->num_experts, a->intermediate_size, kWideWaves * 16,
                    a->hidden_size, a->gate_up.group_size);
  s->act = take(kParts * pairs * s->act_stride * 2);      // float32 ones are smaller
  s->pair_stride = up(a->hidden_size, 16);
  s->pair_out = take(s->wide ? pairs * s->pair_stride * 4 : 0);
  s->total = std::max<int64_t>(off, 256);
  return MOE_EP_OK;
}

}  // namespace

extern "C" {

int moe_ep_route(const moe_ep_router* router, const void* logits, int32_t logits_dtype, int64_t logits_stride,
                 int32_t num_tokens, int32_t* topk_ids, float* topk_weights, void* stream) {
  if (!router) return report(MOE_EP_ERR_INVALID_ARG, "router is NULL");
  if (num_tokens < 0) return report(MOE_EP_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  int st = check_router(*router);
  if (st == MOE_EP_OK) st = check_logits(*router, logits, logits_dtype, logits_stride, num_tokens);
  if (st != MOE_EP_OK) return st;
  if (num_tokens > 0 && (!topk_ids || !topk_weights))
    return report(MOE_EP_ERR_INVALID_ARG, "NULL topk_ids or topk_weights with %d tokens", num_tokens);
  if (!aligned_to(topk_ids, 4) || !aligned_to(topk_weights, 4))
    return report(MOE_EP_ERR_ALIGN, "topk_ids or topk_weights not 4-byte aligned");
  if (num_tokens == 0) return MOE_EP_OK;
  st = check_stream(stream);
  if (st != MOE_EP_OK) return st;
  const hipError_t e = launch_route(
      route_args(*router, logits, logits_dtype, logits_stride, num_tokens, topk_ids, topk_weights),
      static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return report(MOE_EP_ERR_HIP, "route launch failed: %s", hipGetErrorString(e));
  return MOE_EP_OK;
}

int moe_ep_expert_linear(const moe_ep_linear_args* a, void* stream) {
  if (!a) return report(MOE_EP_ERR_INVALID_ARG, "args is NULL");
  int st = check_types(a->dtype, a->out_dtype);
  if (st == MOE_EP_OK) st = check_experts(a->num_experts, a->expert_offset);
  if (st != MOE_EP_OK) return st;
  if (a->num_rows < 0) return report(MOE_EP_ERR_INVALID_ARG, "num_rows %d < 0", a->num_rows);
  if (a->in_features < kMinRow || a->in_features > kMaxSide)
    return report(MOE_EP_ERR_INVALID_ARG, "in_features %d outside [%d, %d]", a->in_features, kMinRow, kMaxSide);
  if (a->out_features < 1 || a->out_features > kMaxSide)
    return report(MOE_EP_ERR_INVALID_ARG, "out_features %d outside [1, %d]", a->out_features, kMaxSide);
  const int out_esz = elem_bytes(a->out_dtype);
  st = check_rows("x", a->x, a->x_stride, a->in_features, a->num_rows, 2, true);
  if (st == MOE_EP_OK) st = check_rows("out", a->out, a->out_stride, a->out_features, a->num_rows, out_esz, false);
  if (st != MOE_EP_OK) return st;
  if (!aligned_to(a->expert_ids, 4)) return report(MOE_EP_ERR_ALIGN, "expert_ids not 4-byte aligned");
  RowsKArgs k = {};
  st = make_weight(a->weight, a->out_features, a->in_features, "weight", &k.w);
  if (st != MOE_EP_OK) return st;
  if (a->num_rows == 0) return MOE_EP_OK;
  if (overlap(a->x, a->x_stride, a->in_features, 2, a->out, a->out_stride, a->out_features, out_esz, a->num_rows))
    return report(MOE_EP_ERR_INVALID_ARG, "x and out overlap");
  st = check_stream(stream);
  if (st != MOE_EP_OK) return st;
  k.x_stride = a->x_stride;
  k.out_stride = a->out_stride;
  k.out_f32 = a->out_dtype == MOE_EP_F32;
  k.top_k = 1;
  k.offset = a->expert_offset;
  k.num_experts = a->num_experts;
  k.inter = a->out_features;
  for (int64_t t = 0; t < a->num_rows; t += kPassTokens) {
    k.n = (int32_t)std::min<int64_t>(kPassTokens, a->num_rows - t);
    k.x = static_cast<const uint16_t*>(a->x) + t * a->x_stride;
    k.out = static_cast<uint8_t*>(a->out) + t * a->out_stride * out_esz;
    k.ids = a->expert_ids ? a->expert_ids + t : nullptr;
    k.by_pair = k.n <= a->num_experts;
    k.wide = is_wide(k.n, 1, k.ids ? a->num_experts : 1, a->out_features, kWideWaves * 32, a->in_features,
                     a->weight.group_size);
    const hipError_t e = launch_expert_linear(k, a->dtype, a->weight.group_size, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return report(MOE_EP_ERR_HIP, "expert_linear launch failed: %s", hipGetErrorString(e));
  }
  return MOE_EP_OK;
}

int moe_ep_layer_workspace_bytes(const moe_ep_layer_args* a, size_t* out_bytes) {
  if (!a || !out_bytes) return report(MOE_EP_ERR_INVALID_ARG, "NULL args or out_bytes");
  LayerSpace s;
  const int st = make_space(a, &s);
  if (st != MOE_EP_OK) return st;
  *out_bytes = (size_t)s.total;
  return MOE_EP_OK;
}

int moe_ep_layer(const moe_ep_layer_args* a, void* stream) {
  if (!a) return report(MOE_EP_ERR_INVALID_ARG, "args is NULL");
  int st = check_types(a->dtype, a->out_dtype);
  if (st != MOE_EP_OK) return st;
  LayerSpace s;
  st = make_space(a, &s);
  if (st != MOE_EP_OK) return st;
  const int n = a->num_tokens;
  const int out_esz = elem_bytes(a->out_dtype);
  st = check_rows("hidden", a->hidden, a->hidden_stride, a->hidden_size, n, 2, true);
  if (st == MOE_EP_OK) st = check_rows("out", a->out, a->out_stride, a->hidden_size, n, out_esz, false);
  if (st != MOE_EP_OK) return st;
  if (a->router) {
    st = check_router(*a->router);
    if (st == MOE_EP_OK) st = check_logits(*a->router, a->router_logits, a->logits_dtype, a->logits_stride, n);
    if (st != MOE_EP_OK) return st;
    if (a->router->top_k != a->top_k)
      return report(MOE_EP_ERR_INVALID_ARG, "top_k %d differs from the router's %d", a->top_k, a->router->top_k);
    if (a->topk_ids || a->topk_weights)
      return report(MOE_EP_ERR_INVALID_ARG, "topk_ids or topk_weights passed together with a router");
  } else {
    if (n > 0 && !a->topk_ids) return report(MOE_EP_ERR_INVALID_ARG, "neither topk_ids nor a router");
    if (!aligned_to(a->topk_ids, 4) || !aligned_to(a->topk_weights, 4))
      return report(MOE_EP_ERR_ALIGN, "topk_ids or topk_weights not 4-byte aligned");
  }
  RowsKArgs r = {};
  DownKArgs d = {};
  st = make_weight(a->gate_up, 2 * (int64_t)a->intermediate_size, a->hidden_size, "gate_up", &r.w);
  if (st == MOE_EP_OK) st = make_weight(a->down, a->hidden_size, a->intermediate_size, "down", &d.w);
  if (st != MOE_EP_OK) return st;
  if (n == 0) return MOE_EP_OK;
  if (overlap(a->hidden, a->hidden_stride, a->hidden_size, 2, a->out, a->out_stride, a->hidden_size, out_esz, n) &&
      !(a->hidden == a->out && a->hidden_stride == a->out_stride && out_esz == 2))
    return report(MOE_EP_ERR_INVALID_ARG, "hidden and out overlap without being the same rows");
  if (!a->workspace || !aligned_to(a->workspace, 256))
    return report(a->workspace ? MOE_EP_ERR_ALIGN : MOE_EP_ERR_INVALID_ARG, "workspace is %s",
                  a->workspace ? "not 256-byte aligned" : "NULL");
  if (a->workspace_bytes < (size_t)s.total)
    return report(MOE_EP_ERR_INVALID_ARG, "workspace has %zu bytes, needs %lld", a->workspace_bytes,
                  (long long)s.total);
  st = check_stream(stream);
  if (st != MOE_EP_OK) return st;

  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  PlanK p;
  p.head = reinterpret_cast<int32_t*>(ws + s.head);
  p.pair = ws + s.pair;
  p.act = ws + s.act;
  p.act_stride = s.act_stride;
  r.x_stride = a->hidden_stride;
  r.top_k = d.top_k = a->top_k;
  r.offset = a->expert_offset;
  r.num_experts = a->num_experts;
  r.inter = a->intermediate_size;
  d.out_stride = a->out_stride;
  d.out_f32 = a->out_dtype == MOE_EP_F32;
  d.tiles = (a->hidden_size + 15) / 16;
  int32_t* ids = reinterpret_cast<int32_t*>(ws + s.ids);
  float* weights = reinterpret_cast<float*>(ws + s.weights);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  for (int64_t t = 0; t < n; t += kPassTokens) {
    const int m = (int)std::min<int64_t>(kPassTokens, n - t);
    const int64_t pairs = (int64_t)m * a->top_k;
    // A few tokens are routed by the first product's kernel itself.
    const bool routed = a->router && !s.wide && m <= kRoutedTokens && pairs <= kFewPairs &&
                        a->router->num_experts <= kRoutedExperts;
    RouteKArgs choice = {};
    if (a->router) {
      const uint8_t* logits =
          static_cast<const uint8_t*>(a->router_logits) + t * a->logits_stride * elem_bytes(a->logits_dtype);
      choice = route_args(*a->router, logits, a->logits_dtype, a->logits_stride, m, ids, weights);
      if (!routed) {
        const hipError_t e = launch_route(choice, hs);
        if (e != hipSuccess) return report(MOE_EP_ERR_HIP, "route launch failed: %s", hipGetErrorString(e));
      }
    }
    r.n = d.n = m;
    r.x = static_cast<const uint16_t*>(a->hidden) + t * a->hidden_stride;
    r.ids = a->router ? ids : a->topk_ids + t * a->top_k;
    r.topk_weights = a->router ? weights : a->topk_weights ? a->topk_weights + t * a->top_k : nullptr;
    r.by_pair = pairs <= a->num_experts;
    p.slots = (int32_t)std::min<int64_t>(pairs, a->num_experts);
    p.act_plane = s.wide || a->down.group_size ? pairs * p.act_stride : 0;
    r.plan = d.plan = p;
    d.out = static_cast<uint8_t*>(a->out) + t * a->out_stride * out_esz;
    d.chunks = (m + kChunkTokens - 1) / kChunkTokens;
    r.wide = s.wide;
    hipError_t e;
    if (routed) {
      RowsRoutedKArgs rr;
      static_cast<RowsKArgs&>(rr) = r;
      rr.route = choice;
      e = launch_gate_up_routed(rr, a->dtype, a->gate_up.group_size, hs);
    } else {
      e = launch_gate_up(r, a->dtype, a->gate_up.group_size, hs);
    }
    if (e == hipSuccess && s.wide) {
      RowsKArgs y = r;
      y.w = d.w;
      y.inter = a->hidden_size;
      y.pair_out = reinterpret_cast<float*>(ws + s.pair_out);
      y.pair_stride = s.pair_stride;
      y.out = d.out;
      y.out_stride = d.out_stride;
      y.out_f32 = d.out_f32;
      e = launch_wide_down(y, a->dtype, a->down.group_size, hs);
    } else if (e == hipSuccess) {
      e = launch_down(d, a->dtype, a->down.group_size, hs);
    }
    if (e != hipSuccess) return report(MOE_EP_ERR_HIP, "layer launch failed: %s", hipGetErrorString(e));
  }
  return MOE_EP_OK;
}

}  // extern "C"
