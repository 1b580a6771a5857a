// C-ABI host side of the dense operators: argument checks and launches.
// Every check comes before the first launch, so a refused call leaves no
// device work behind.

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "moe_args_internal.h"
#include "moe_dense_internal.h"
#include "moe_ep.h"

using namespace moe_ep_detail;

namespace {

// A set of rows of one call, for checks against the others.
struct RowSet {
  const char* what;
  const void* p;
  int64_t stride, width;
  int esz;
  int n;
};

bool meet(const RowSet& a, const RowSet& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + (uintptr_t)(((a.n - 1) * a.stride + a.width) * a.esz);
  const uintptr_t b1 = b0 + (uintptr_t)(((b.n - 1) * b.stride + b.width) * b.esz);
  return a0 < b1 && b0 < a1;
}

bool same_rows(const RowSet& a, const RowSet& b) {
  return a.p == b.p && a.esz == b.esz && (a.stride == b.stride || a.n <= 1);
}

// Refuses an output that meets an input or another output.
int check_apart(const RowSet* in, int ins, const RowSet* out, int outs) {
  for (int o = 0; o < outs; ++o) {
    for (int i = 0; i < ins; ++i)
      if (meet(out[o], in[i]))
        return report(MOE_EP_ERR_INVALID_ARG, "%s and %s overlap", out[o].what, in[i].what);
    for (int p = 0; p < o; ++p)
      if (meet(out[o], out[p])) return report(MOE_EP_ERR_INVALID_ARG, "%s and %s overlap", out[o].what, out[p].what);
  }
  return MOE_EP_OK;
}

int check_side(const char* what, int64_t v, int64_t least) {
  if (v < least || v > kMaxSide)
    return report(MOE_EP_ERR_INVALID_ARG, "%s %lld outside [%lld, %d]", what, (long long)v, (long long)least, kMaxSide);
  return MOE_EP_OK;
}

int check_workspace(const void* p, size_t have, size_t need) {
  if (!p) return report(MOE_EP_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned_to(p, 256)) return report(MOE_EP_ERR_ALIGN, "workspace is not 256-byte aligned");
  if (have < need) return report(MOE_EP_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", have, need);
  return MOE_EP_OK;
}

// A launch has fewer than 2^32 threads: 512 for each tile of 128 x 128 results
// (smaller ones are for fewer results).
int check_tiles(int64_t rows, int64_t cols) {
  if ((rows + 127) / 128 * ((cols + 127) / 128) >= 1 << 23)
    return report(MOE_EP_ERR_INVALID_ARG, "%lld x %lld results are 2^23 tiles of 128 x 128 or more", (long long)rows,
                  (long long)cols);
  return MOE_EP_OK;
}

// An operand of the products; `side` is its extent that lies side by side.
MatK operand(const void* p, int64_t stride, int32_t rows, int64_t side) {
  MatK m;
  m.p = static_cast<const uint16_t*>(p);
  m.stride = stride;
  m.rows = rows;
  m.whole = aligned_to(p, 16) && stride % 8 == 0 && stride <= kMaxSide && side % 8 == 0;
  return m;
}

// Workspace of the gated product's gradients: [d][rest of d, with two
// parts][tops][factor][partial sums].
struct GradSpace {
  int64_t d_stride, rest, tops, factor, partial, total;
};

int make_space(const moe_ep_gated_grad_args* a, GradSpace* s) {
  if (a->dtype != MOE_EP_BF16 && a->dtype != MOE_EP_F16)
    return report(MOE_EP_ERR_INVALID_ARG, "dtype %d is not MOE_EP_BF16 or MOE_EP_F16", a->dtype);
  if (a->num_rows < 0) return report(MOE_EP_ERR_INVALID_ARG, "num_rows %d < 0", a->num_rows);
  int st = check_side("hidden_size", a->hidden_size, kMinRow);
  if (st == MOE_EP_OK) st = check_side("intermediate_size", a->intermediate_size, kMinRow);
  if (st != MOE_EP_OK) return st;
  if (a->d_parts < 0 || a->d_parts > 2)
    return report(MOE_EP_ERR_INVALID_ARG, "d_parts %d is not 0, 1 or 2", a->d_parts);
  s->d_stride = up(2 * (int64_t)a->intermediate_size, 8);
  s->rest = up(a->num_rows * s->d_stride * 2, 256);
  s->tops = a->d_parts == 2 ? 2 * s->rest : s->rest;
  s->factor = s->tops + (a->dtype == MOE_EP_F16 ? kTops * 4 : 0);
  s->partial = s->factor + 256;
  s->total = s->partial + kPartialFloats * 4;
  return MOE_EP_OK;
}

// Rows of an adapter_linear call: its first kernel has 64 threads for each.
constexpr int32_t kMaxAdapterRows = 1 << 25;

int check_adapter_sizes(const moe_ep_adapter_args* a) {
  if (a->num_rows < 0 || a->num_rows > kMaxAdapterRows)
    return report(MOE_EP_ERR_INVALID_ARG, "num_rows %d outside [0, %d]", a->num_rows, kMaxAdapterRows);
  if (a->num_adapters < 1 || a->num_adapters > MOE_EP_MAX_EXPERTS)
    return report(MOE_EP_ERR_INVALID_ARG, "num_adapters %d outside [1, %d]", a->num_adapters, MOE_EP_MAX_EXPERTS);
  if (a->rank < 1 || a->rank > MOE_EP_MAX_RANK)
    return report(MOE_EP_ERR_INVALID_ARG, "rank %d outside [1, %d]", a->rank, MOE_EP_MAX_RANK);
  const int st = check_side("in_features", a->in_features, kMinRow);
  return st != MOE_EP_OK ? st : check_side("out_features", a->out_features, 1);
}

size_t adapter_workspace(const moe_ep_adapter_args* a) {
  return std::max<size_t>((size_t)up(LowSpace(a->num_rows, a->rank).bytes, 256), 256);
}

}  // namespace

extern "C" {

int moe_ep_rms_norm(const moe_ep_norm_args* a, void* stream) {
  if (!a) return report(MOE_EP_ERR_INVALID_ARG, "args is NULL");
  if (a->dtype != MOE_EP_BF16 && a->dtype != MOE_EP_F16)
    return report(MOE_EP_ERR_INVALID_ARG, "dtype %d is not MOE_EP_BF16 or MOE_EP_F16", a->dtype);
  if (a->weight_dtype != a->dtype && a->weight_dtype != MOE_EP_F32)
    return report(MOE_EP_ERR_INVALID_ARG, "weight_dtype %d is neither dtype %d nor MOE_EP_F32", a->weight_dtype,
                  a->dtype);
  const bool eight = a->out_dtype == MOE_EP_E4M3;
  if (!eight && a->out_dtype != a->dtype)
    return report(MOE_EP_ERR_INVALID_ARG, "out_dtype %d is neither dtype %d nor MOE_EP_E4M3", a->out_dtype, a->dtype);
  const int g = a->group_size, n = a->num_rows;
  if (g != 0 && (!eight || (g != 32 && g != 64 && g != 128)))
    return report(MOE_EP_ERR_INVALID_ARG, "group_size %d is not 0%s", g, eight ? ", 32, 64 or 128" : " for 16-bit rows");
  if (n < 0) return report(MOE_EP_ERR_INVALID_ARG, "num_rows %d < 0", n);
  const int H = a->hidden_size;
  if (H < kMinRow || H > kMaxSide)
    return report(MOE_EP_ERR_INVALID_ARG, "hidden_size %d outside [%d, %d]", H, kMinRow, kMaxSide);
  if (!(a->eps >= 0) || !std::isfinite(a->eps))
    return report(MOE_EP_ERR_INVALID_ARG, "eps %g is not finite and >= 0", (double)a->eps);
  const int groups = g ? (H + g - 1) / g : 1;
  int st = check_rows("x", a->x, a->x_stride, H, n, 2, true);
  if (st == MOE_EP_OK && a->residual) st = check_rows("residual", a->residual, a->residual_stride, H, n, 2, true);
  if (st == MOE_EP_OK) st = check_rows("out", a->out, a->out_stride, H, n, eight ? 1 : 2, false);
  if (st == MOE_EP_OK && a->residual_out)
    st = check_rows("residual_out", a->residual_out, a->residual_out_stride, H, n, 2, false);
  if (st == MOE_EP_OK && eight) st = check_rows("scales", a->scales, a->scales_stride, groups, n, 4, false);
  if (st != MOE_EP_OK) return st;
  if (a->residual_out && !a->residual)
    return report(MOE_EP_ERR_INVALID_ARG, "residual_out without residual");
  if (!eight && a->scales) return report(MOE_EP_ERR_INVALID_ARG, "scales with 16-bit rows");
  if (!a->weight) return report(MOE_EP_ERR_INVALID_ARG, "weight is NULL");
  if (!aligned_to(a->weight, a->weight_dtype == MOE_EP_F32 ? 4 : 2))
    return report(MOE_EP_ERR_ALIGN, "weight not aligned to its element");
  if (n == 0) return MOE_EP_OK;
  const RowSet in[] = {{"x", a->x, a->x_stride, H, 2, n},
                       {"residual", a->residual, a->residual_stride, H, 2, n},
                       {"weight", a->weight, 0, H, a->weight_dtype == MOE_EP_F32 ? 4 : 2, 1}};
  const RowSet out[] = {{"out", a->out, a->out_stride, H, eight ? 1 : 2, n},
                        {"residual_out", a->residual_out, a->residual_out_stride, H, 2, n},
                        {"scales", a->scales, a->scales_stride, groups, 4, eight ? n : 0}};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 3; ++i)
      if (meet(out[o], in[i]) && !(o < 2 && i < 2 && same_rows(out[o], in[i])))
        return report(MOE_EP_ERR_INVALID_ARG, "%s and %s overlap without being the same rows", out[o].what, in[i].what);
    for (int p = 0; p < o; ++p)
      if (meet(out[o], out[p])) return report(MOE_EP_ERR_INVALID_ARG, "%s and %s overlap", out[o].what, out[p].what);
  }
  st = check_stream(stream);
  if (st != MOE_EP_OK) return st;
  NormKArgs k;
  k.x = static_cast<const uint16_t*>(a->x);
  k.residual = static_cast<const uint16_t*>(a->residual);
  k.weight = a->weight;
  k.out = a->out;
  k.scales = a->scales;
  k.residual_out = static_cast<uint16_t*>(a->residual_out);
  k.x_stride = a->x_stride;
  k.residual_stride = a->residual_stride;
  k.out_stride = a->out_stride;
  k.scales_stride = a->scales_stride;
  k.residual_out_stride = a->residual_out_stride;
  k.n = n;
  k.hidden = H;
  k.group = g;
  k.eps = a->eps;
  const hipError_t e =
      launch_rms_norm(k, a->dtype, a->weight_dtype == MOE_EP_F32, eight, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return report(MOE_EP_ERR_HIP, "rms_norm launch failed: %s", hipGetErrorString(e));
  return MOE_EP_OK;
}

int moe_ep_gated(const moe_ep_gated_args* a, void* stream) {
  if (!a) return report(MOE_EP_ERR_INVALID_ARG, "args is NULL");
  int st = check_types(a->dtype, a->out_dtype);
  if (st != MOE_EP_OK) return st;
  const int n = a->num_rows, H = a->hidden_size, I = a->intermediate_size;
  if (n < 0) return report(MOE_EP_ERR_INVALID_ARG, "num_rows %d < 0", n);
  st = check_side("hidden_size", H, kMinRow);
  if (st == MOE_EP_OK) st = check_side("intermediate_size", I, kMinRow);
  if (st == MOE_EP_OK) st = check_tiles(n, 2 * (int64_t)I);
  const int out_esz = elem_bytes(a->out_dtype);
  if (st == MOE_EP_OK) st = check_rows("x", a->x, a->x_stride, H, n, 2, true);
  if (st == MOE_EP_OK) st = check_rows("gate_up", a->gate_up, a->gate_up_stride, H, 2 * I, 2, false);
  if (st == MOE_EP_OK) st = check_rows("out", a->out, a->out_stride, I, n, out_esz, false);
  if (st != MOE_EP_OK) return st;
  if (!aligned_to(a->pre, 4)) return report(MOE_EP_ERR_ALIGN, "pre not aligned to its element");
  if (n == 0) return MOE_EP_OK;
  const RowSet in[] = {{"x", a->x, a->x_stride, H, 2, n}, {"gate_up", a->gate_up, a->gate_up_stride, H, 2, 2 * I}};
  const RowSet out[] = {{"out", a->out, a->out_stride, I, out_esz, n},
                        {"pre", a->pre, 2 * (int64_t)I, 2 * (int64_t)I, 4, n}};
  st = check_apart(in, 2, out, 2);
  if (st == MOE_EP_OK) st = check_stream(stream);
  if (st != MOE_EP_OK) return st;
  GatedKArgs k = {};
  k.w = operand(a->gate_up, a->gate_up_stride, I, H);
  k.x = operand(a->x, a->x_stride, n, H);
  k.hidden = H;
  k.inter = I;
  k.out = a->out;
  k.pre = a->pre;
  k.out_stride = a->out_stride;
  k.out_f32 = a->out_dtype == MOE_EP_F32;
  const hipError_t e = launch_gated(k, a->dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return report(MOE_EP_ERR_HIP, "gated launch failed: %s", hipGetErrorString(e));
  return MOE_EP_OK;
}

int moe_ep_gated_grad_workspace_bytes(const moe_ep_gated_grad_args* a, size_t* out_bytes) {
  if (!a || !out_bytes) return report(MOE_EP_ERR_INVALID_ARG, "NULL args or out_bytes");
  GradSpace s;
  const int st = make_space(a, &s);
  if (st != MOE_EP_OK) return st;
  *out_bytes = (size_t)s.total;
  return MOE_EP_OK;
}

int moe_ep_gated_grad(const moe_ep_gated_grad_args* a, void* stream) {
  if (!a) return report(MOE_EP_ERR_INVALID_ARG, "args is NULL");
  int st = check_types(a->dtype, a->dout_dtype);
  GradSpace s;
  if (st == MOE_EP_OK) st = make_space(a, &s);
  if (st != MOE_EP_OK) return st;
  const int n = a->num_rows, H = a->hidden_size, I = a->intermediate_size;
  const bool half = a->dtype == MOE_EP_F16;
  const int dout_esz = elem_bytes(a->dout_dtype);
  st = check_tiles(n, H);
  if (st == MOE_EP_OK) st = check_tiles(2 * (int64_t)I, H);
  if (st == MOE_EP_OK) st = check_rows("dout", a->dout, a->dout_stride, I, n, dout_esz, true);
  if (st == MOE_EP_OK && a->dgate_up) st = check_rows("x", a->x, a->x_stride, H, n, 2, true);
  if (st == MOE_EP_OK && a->dx) st = check_rows("gate_up", a->gate_up, a->gate_up_stride, H, 2 * I, 2, false);
  if (st == MOE_EP_OK && a->dx) st = check_rows("dx", a->dx, a->dx_stride, H, n, 2, false);
  if (st == MOE_EP_OK && a->dgate_up)
    st = check_rows("dgate_up", a->dgate_up, a->dgate_up_stride, H, 2 * I, 2, false);
  if (st != MOE_EP_OK) return st;
  if (n > 0 && !a->pre) return report(MOE_EP_ERR_INVALID_ARG, "pre is NULL with %d rows", n);
  if (!aligned_to(a->pre, 4)) return report(MOE_EP_ERR_ALIGN, "pre not aligned to its element");
  if ((!a->dx || n == 0) && !a->dgate_up) return MOE_EP_OK;
  st = check_workspace(a->workspace, a->workspace_bytes, (size_t)s.total);
  if (st != MOE_EP_OK) return st;
  const RowSet in[] = {{"dout", a->dout, a->dout_stride, I, dout_esz, n},
                       {"x", a->dgate_up ? a->x : nullptr, a->x_stride, H, 2, n},
                       {"gate_up", a->dx ? a->gate_up : nullptr, a->gate_up_stride, H, 2, 2 * I},
                       {"pre", a->pre, 2 * (int64_t)I, 2 * (int64_t)I, 4, n}};
  const RowSet out[] = {{"dx", a->dx, a->dx_stride, H, 2, n},
                        {"dgate_up", a->dgate_up, a->dgate_up_stride, H, 2, 2 * I},
                        {"workspace", a->workspace, 0, s.total, 1, 1}};
  st = check_apart(in, 4, out, 3);
  if (st == MOE_EP_OK) st = check_stream(stream);
  if (st != MOE_EP_OK) return st;

  hipStream_t hs = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  uint16_t* d = reinterpret_cast<uint16_t*>(ws);
  uint16_t* rest = a->d_parts == 2 && n > 0 ? reinterpret_cast<uint16_t*>(ws + s.rest) : nullptr;
  hipError_t e = hipSuccess;
  ProductKArgs k = {};
  k.partial = reinterpret_cast<float*>(ws + s.partial);
  k.q_rest = rest ? rest - d : 0;
  if (n > 0) {
    GatedGradKArgs g = {};
    g.dout = a->dout;
    g.pre = a->pre;
    g.d = d;
    g.rest = rest;
    g.dout_stride = a->dout_stride;
    g.d_stride = s.d_stride;
    g.dout_f32 = a->dout_dtype == MOE_EP_F32;
    g.n = n;
    g.inter = I;
    g.tops = half ? reinterpret_cast<uint32_t*>(ws + s.tops) : nullptr;
    g.factor = half ? reinterpret_cast<float*>(ws + s.factor) : nullptr;
    k.factor = g.factor;
    e = launch_gated_grad(g, a->dtype, hs);
  }
  if (e == hipSuccess && a->dx && n > 0) {
    k.p = operand(a->gate_up, a->gate_up_stride, H, H);
    k.q = operand(d, s.d_stride, n, s.d_stride);
    k.p.whole = k.p.whole && 2 * (int64_t)I % 8 == 0;     // the products end with k in both operands
    k.k = 2 * I;
    k.q_rows = n;
    k.out = static_cast<uint16_t*>(a->dx);
    k.out_stride = a->dx_stride;
    e = launch_product(k, a->dtype, true, hs);
  }
  if (e == hipSuccess && a->dgate_up) {
    k.p = operand(a->x, a->x_stride, H, H);
    k.q = operand(d, s.d_stride, (int32_t)s.d_stride, s.d_stride);
    k.k = n;
    k.q_rows = 2 * I;
    k.out = static_cast<uint16_t*>(a->dgate_up);
    k.out_stride = a->dgate_up_stride;
    e = launch_product(k, a->dtype, false, hs);
  }
  if (e != hipSuccess) return report(MOE_EP_ERR_HIP, "gated_grad launch failed: %s", hipGetErrorString(e));
  return MOE_EP_OK;
}

int moe_ep_adapter_workspace_bytes(const moe_ep_adapter_args* a, size_t* out_bytes) {
  if (!a || !out_bytes) return report(MOE_EP_ERR_INVALID_ARG, "NULL args or out_bytes");
  const int st = check_adapter_sizes(a);
  if (st != MOE_EP_OK) return st;
  *out_bytes = adapter_workspace(a);
  return MOE_EP_OK;
}

int moe_ep_adapter_linear(const moe_ep_adapter_args* a, void* stream) {
  if (!a) return report(MOE_EP_ERR_INVALID_ARG, "args is NULL");
  int st = check_types(a->dtype, a->out_dtype);
  if (st == MOE_EP_OK) st = check_adapter_sizes(a);
  if (st != MOE_EP_OK) return st;
  const int n = a->num_rows, N = a->out_features, K = a->in_features;
  const int64_t L = a->num_adapters, R = a->rank;
  const int out_esz = elem_bytes(a->out_dtype);
  st = check_tiles(n, N);
  if (st == MOE_EP_OK) st = check_rows("x", a->x, a->x_stride, K, n, 2, true);
  if (st == MOE_EP_OK) st = check_rows("weight", a->weight, a->weight_stride, K, N, 2, false);
  if (st == MOE_EP_OK) st = check_rows("lora_a", a->lora_a, K, K, 1, 2, false);
  if (st == MOE_EP_OK) st = check_rows("lora_b", a->lora_b, R, R, 1, 2, false);
  if (st == MOE_EP_OK) st = check_rows("out", a->out, a->out_stride, N, n, out_esz, false);
  if (st != MOE_EP_OK) return st;
  if (n > 0 && !a->adapter_ids) return report(MOE_EP_ERR_INVALID_ARG, "adapter_ids is NULL with %d rows", n);
  if (!aligned_to(a->adapter_ids, 4) || !aligned_to(a->scales, 4))
    return report(MOE_EP_ERR_ALIGN, "adapter_ids or scales not 4-byte aligned");
  if (n == 0) return MOE_EP_OK;
  const size_t need = adapter_workspace(a);
  st = check_workspace(a->workspace, a->workspace_bytes, need);
  if (st != MOE_EP_OK) return st;
  const RowSet in[] = {{"x", a->x, a->x_stride, K, 2, n},
                       {"weight", a->weight, a->weight_stride, K, 2, N},
                       {"lora_a", a->lora_a, 0, L * R * K, 2, 1},
                       {"lora_b", a->lora_b, 0, L * R * N, 2, 1},
                       {"adapter_ids", a->adapter_ids, 0, n, 4, 1},
                       {"scales", a->scales, 0, L, 4, 1}};
  const RowSet out[] = {{"out", a->out, a->out_stride, N, out_esz, n},
                        {"workspace", a->workspace, 0, (int64_t)need, 1, 1}};
  st = check_apart(in, 6, out, 2);
  if (st == MOE_EP_OK) st = check_stream(stream);
  if (st != MOE_EP_OK) return st;

  AdapterKArgs k = {};
  k.w = operand(a->weight, a->weight_stride, N, K);
  k.x = operand(a->x, a->x_stride, n, K);
  k.k = K;
  k.out = a->out;
  k.out_stride = a->out_stride;
  k.out_f32 = a->out_dtype == MOE_EP_F32;
  k.a = static_cast<const uint16_t*>(a->lora_a);
  k.low = a->workspace;
  k.low_stride = LowSpace(n, a->rank).stride;
  k.b = static_cast<const uint16_t*>(a->lora_b);
  k.ids = a->adapter_ids;
  k.scales = a->scales;
  k.adapters = a->num_adapters;
  k.rank = a->rank;
  const hipError_t e = launch_adapter(k, a->dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return report(MOE_EP_ERR_HIP, "adapter_linear launch failed: %s", hipGetErrorString(e));
  return MOE_EP_OK;
}

}  // extern "C"
