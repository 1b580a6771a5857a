"""What a block computes on all of its tokens beside the routed experts, over
torch tensors:

* ``rms_norm``        the residual's addition and a root-mean-square norm, in
                      16 bits or in 8 bits with scales as dispatch takes them
* ``gated_linear``    the first half of a gated feed-forward (a shared
                      expert's), with its backward pass
* ``adapter_linear``  a projection that all rows share, with a low-rank
                      adapter of each row's own

Every step runs in the library's gfx950 kernels (include/moe_ep.h); torch is
used for device memory and the current stream.  Work is enqueued on the
current stream of the tensors' device; what a call needs beyond its inputs
comes from torch's allocator for that stream, so calls may be captured into
graphs and run on several streams at once.  Tensors that carry a forward-mode
derivative are refused.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from .experts import (_DTYPES, _activations, _call, _forward_only, _ids, _int32, _no_tangents, _on, _output,
                      _rows, _written)


@dataclass
class NormResult:
    """What ``rms_norm`` made of its rows."""

    rows: torch.Tensor                      # [n, hidden] of x's type, or float8_e4m3fn
    scales: Optional[torch.Tensor]          # float32 [n, groups] of 8-bit rows, else None
    residual: Optional[torch.Tensor]        # [n, hidden], x + residual; None without a residual


def _result(out: Optional[torch.Tensor], shape, dtype: torch.dtype, x: torch.Tensor, dev: int, what: str):
    """(tensor, address, row stride) of ``out``, checked, or of a new tensor
    (one of x's shape is made in half the time of any other)."""
    if out is None:
        out = torch.empty_like(x, dtype=dtype) if shape == x.shape else x.new_empty(shape, dtype=dtype)
        return out, out.data_ptr(), out.stride(0)
    if out.dtype != dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{what} must be {dtype} {list(shape)}")
    return (out, *_rows(out, dev, what))


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
             out_dtype: Optional[torch.dtype] = None, group_size: int = 0, out: Optional[torch.Tensor] = None,
             scales: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None) -> NormResult:
    """``s / sqrt(mean(s * s) + eps) * weight`` of each row of ``s = x +
    residual``, and ``s`` as the new residual.

    ``x`` and ``residual`` [rows, hidden] are bfloat16 or float16 (rows may be
    strided), ``weight`` [hidden] is of their type or float32.  The rows come
    in x's type, or with ``out_dtype=torch.float8_e4m3fn`` in 8 bits: then
    ``scales`` (float32) holds max / 448 of each ``group_size`` (32, 64 or
    128) columns, 0: of a whole row, and rows times scales are the values.
    Rows and scales are what ``MoEEp.dispatch`` takes as hidden rows and
    ``hidden_states_scale``.

    ``out`` and ``residual_out`` may be ``x`` or ``residual`` themselves;
    ``residual_out=residual`` updates it in place.  There is no backward pass.
    See include/moe_ep.h, moe_ep_rms_norm."""
    _forward_only("rms_norm", x, weight, residual, out, scales, residual_out)
    dev = _activations(x, "x")
    n, H = x.shape
    a = _lib.moe_ep_norm_args()
    given = (out, scales, residual_out)
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        raise TypeError(f"weight is {weight.dtype}, x {x.dtype}: it must be of x's type or float32")
    if tuple(weight.shape) != (H,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous [{H}]")
    eight = out_dtype == torch.float8_e4m3fn
    if not eight and out_dtype is not None and out_dtype != x.dtype:
        raise TypeError(f"out_dtype must be {x.dtype} or torch.float8_e4m3fn, got {out_dtype}")
    odt = torch.float8_e4m3fn if eight else x.dtype
    a.x, a.x_stride = _rows(x, dev, "x")
    out, a.out, a.out_stride = _result(out, (n, H), odt, x, dev, "out")
    a.weight = _on(weight, dev, "weight")
    if eight:
        if group_size not in (0, 32, 64, 128):
            raise ValueError(f"group_size {group_size} is not 0, 32, 64 or 128")
        shape = (n, -(-H // group_size) if group_size else 1)
        scales, a.scales, a.scales_stride = _result(scales, shape, torch.float32, x, dev, "scales")
    elif scales is not None or group_size:
        raise ValueError("scales and group_size go with out_dtype=torch.float8_e4m3fn")
    if residual is not None:
        if residual.dtype != x.dtype or residual.shape != x.shape:
            raise ValueError(f"residual must be {x.dtype} {list(x.shape)}")
        a.residual, a.residual_stride = _rows(residual, dev, "residual")
        residual_out, a.residual_out, a.residual_out_stride = _result(residual_out, (n, H), x.dtype, x, dev,
                                                                      "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out goes with residual")
    a.dtype, a.weight_dtype = _DTYPES[x.dtype], _DTYPES[weight.dtype]
    a.out_dtype = _lib.MOE_EP_E4M3 if eight else a.dtype
    a.group_size, a.num_rows, a.hidden_size, a.eps = group_size, _int32(n, "row count"), _int32(H, "hidden size"), eps
    _call(_lib.moe_ep_rms_norm, dev, a)
    _written(*given)
    return NormResult(out, scales, residual_out)


def _matrix(w: torch.Tensor, dev: int, dtype: torch.dtype, cols: int, what: str):
    """Address and row stride of a weight matrix [rows, cols]."""
    if w.dim() != 2 or w.shape[1] != cols:
        raise ValueError(f"{what} must be [rows, {cols}]")
    if w.dtype != dtype:
        raise TypeError(f"{what} is {w.dtype}, the activations {dtype}")
    p, stride = _rows(w, dev, what)
    return p, max(stride, cols) if w.shape[0] <= 1 else stride


def _gated(x: torch.Tensor, gate_up: torch.Tensor, out, out_dtype, keep: bool):
    """(h, pre or None)."""
    dev = _activations(x, "x")
    n, H = x.shape
    a = _lib.moe_ep_gated_args()
    a.gate_up, a.gate_up_stride = _matrix(gate_up, dev, x.dtype, H, "gate_up")
    if gate_up.shape[0] % 2:
        raise ValueError(f"gate_up has {gate_up.shape[0]} rows, not twice as many as the result has columns")
    inter = gate_up.shape[0] // 2
    given, out = out, _output(out, (n, inter), x.dtype, out_dtype, x)
    a.x, a.x_stride = _rows(x, dev, "x")
    a.out, a.out_stride = _rows(out, dev, "out")
    pre = None
    if keep:
        pre = x.new_empty((n, 2 * inter), dtype=torch.float32)
        a.pre = pre.data_ptr()
    a.dtype, a.out_dtype = _DTYPES[x.dtype], _DTYPES[out.dtype]
    a.num_rows, a.hidden_size = _int32(n, "row count"), _int32(H, "hidden size")
    a.intermediate_size = _int32(inter, "intermediate size")
    _call(_lib.moe_ep_gated, dev, a)
    _written(given)
    return out, pre


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate_up, out_dtype, grad_parts):
        h, pre = _gated(x, gate_up, None, out_dtype, True)
        ctx.grad_parts = grad_parts
        ctx.save_for_backward(x, gate_up, pre)
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x, gate_up, pre = ctx.saved_tensors
        dev = x.get_device()
        n, H = x.shape
        inter = gate_up.shape[0] // 2
        if dh.stride(1) != 1 or dh.stride(0) < inter and dh.stride(0) != 0:
            dh = dh.contiguous()                     # an expanded sum's, or a transposed one
        a = _lib.moe_ep_gated_grad_args()
        a.dout, a.dout_stride = _rows(dh, dev, "the gradient")
        a.x, a.x_stride = _rows(x, dev, "x")
        a.gate_up, a.gate_up_stride = _matrix(gate_up, dev, x.dtype, H, "gate_up")
        a.pre = pre.data_ptr()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = x.new_empty((n, H))
            a.dx, a.dx_stride = dx.data_ptr(), H
        if ctx.needs_input_grad[1]:
            dw = x.new_empty((2 * inter, H))
            a.dgate_up, a.dgate_up_stride = dw.data_ptr(), H
        a.dtype, a.dout_dtype = _DTYPES[x.dtype], _DTYPES[dh.dtype]
        a.num_rows, a.hidden_size, a.intermediate_size, a.d_parts = n, H, inter, ctx.grad_parts
        nbytes = _lib.moe_ep_gated_grad_workspace_bytes(a)
        workspace = x.new_empty((nbytes,), dtype=torch.uint8)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), nbytes
        _call(_lib.moe_ep_gated_grad, dev, a)
        return dx, dw, None, None


def gated_linear(x: torch.Tensor, gate_up: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                 out_dtype: Optional[torch.dtype] = None, grad_parts: int = 1) -> torch.Tensor:
    """``silu(x @ gate.T) * (x @ up.T)``: the first half of a gated
    feed-forward, such as a shared expert's.

    ``x`` [rows, hidden] is bfloat16 or float16 (rows may be strided),
    ``gate_up`` [2 * intermediate, hidden] of its type holds the gate rows,
    then the up rows, as ``moe_layer`` takes them for each expert.  The
    result [rows, intermediate] is of x's type or float32 (``out_dtype``).

    Where autograd records (x or gate_up requires gradients), both get theirs,
    in x's type and from float32 sums; gate and up are kept for it as float32
    [rows, 2 * intermediate], and ``out`` is refused.  The gradients of gate
    and up enter the products that make those of x and gate_up in x's type.
    ``grad_parts=1`` rounds them once, as a chain of torch's operators would:
    the results are then off by 1.4 times what their own rounding makes
    (bfloat16 0.0023 of the norm for 0.0017).  ``grad_parts=2`` keeps what that
    rounding leaves as a second number of x's type, and the results are as near
    as their type allows, at twice the products.  As for torch's own
    operators, a ``backward()`` may be captured into a graph only while no
    result that was recorded outside the capture from the same leaves is
    alive: torch would accumulate on the other stream.  See include/moe_ep.h,
    moe_ep_gated and moe_ep_gated_grad."""
    _no_tangents("gated_linear", x, gate_up, out)
    if grad_parts not in (1, 2):
        raise ValueError(f"grad_parts must be 1 or 2, got {grad_parts}")
    if torch.is_grad_enabled() and (x.requires_grad or gate_up.requires_grad or
                                    (out is not None and out.requires_grad)):
        if out is not None:
            raise RuntimeError("gated_linear does not write into out where autograd records: "
                               "call it under torch.no_grad() or without out")
        return _GatedLinear.apply(x, gate_up, out_dtype, grad_parts)
    return _gated(x, gate_up, out, out_dtype, False)[0]


def adapter_linear(x: torch.Tensor, weight: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                   adapter_ids: torch.Tensor, *, scales: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``weight @ x[r] + scales[a] * lora_b[a] @ (lora_a[a] @ x[r])`` with
    ``a = adapter_ids[r]``: a projection that all rows share, each row with
    the low-rank adapter of its request.

    ``x`` [rows, in] is bfloat16 or float16 (rows may be strided), ``weight``
    [out, in], ``lora_a`` [adapters, rank, in] and ``lora_b`` [adapters, out,
    rank] of its type, ``adapter_ids`` int32 or int64 [rows]: a row whose id
    is outside [0, adapters) has no adapter.  ``scales`` is float32
    [adapters]; None: all 1.  Adapters of a smaller rank are padded with
    zeros.  The result is of x's type or float32 (``out_dtype``).

    ``workspace`` (uint8, ``adapter_linear_workspace_bytes`` of it) is taken
    from torch's allocator when not passed; one that is passed must not be
    used by two calls that may overlap in time.  There is no backward pass.
    See include/moe_ep.h, moe_ep_adapter_linear."""
    _forward_only("adapter_linear", x, weight, lora_a, lora_b, scales, out)
    dev = _activations(x, "x")
    n, K = x.shape
    a = _lib.moe_ep_adapter_args()
    a.weight, a.weight_stride = _matrix(weight, dev, x.dtype, K, "weight")
    N = weight.shape[0]
    for t, what in ((lora_a, "lora_a"), (lora_b, "lora_b")):
        if t.dtype != x.dtype:
            raise TypeError(f"{what} is {t.dtype}, the activations {x.dtype}")
    if lora_a.dim() != 3 or lora_a.shape[2] != K or not lora_a.is_contiguous():
        raise ValueError(f"lora_a must be a contiguous [adapters, rank, {K}]")
    L, R = lora_a.shape[0], lora_a.shape[1]
    if tuple(lora_b.shape) != (L, N, R) or not lora_b.is_contiguous():
        raise ValueError(f"lora_b must be a contiguous [{L}, {N}, {R}]")
    a.lora_a, a.lora_b = _on(lora_a, dev, "lora_a"), _on(lora_b, dev, "lora_b")
    adapter_ids = _ids(adapter_ids, (n,), dev, "adapter_ids")
    a.adapter_ids = adapter_ids.data_ptr()
    if scales is not None:
        if scales.dtype != torch.float32 or tuple(scales.shape) != (L,) or not scales.is_contiguous():
            raise ValueError(f"scales must be a contiguous float32 [{L}]")
        a.scales = _on(scales, dev, "scales")
    given, out = out, _output(out, (n, N), x.dtype, out_dtype, x)
    a.x, a.x_stride = _rows(x, dev, "x")
    a.out, a.out_stride = _rows(out, dev, "out")
    a.dtype, a.out_dtype = _DTYPES[x.dtype], _DTYPES[out.dtype]
    a.num_rows = _int32(n, "row count")
    a.in_features, a.out_features = _int32(K, "in_features"), _int32(N, "out_features")
    a.num_adapters, a.rank = _int32(L, "adapter count"), _int32(R, "rank")
    if workspace is None:
        nbytes = _lib.moe_ep_adapter_workspace_bytes(a)
        workspace = x.new_empty((nbytes,), dtype=torch.uint8)
    else:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        nbytes = workspace.numel()
    a.workspace, a.workspace_bytes = _on(workspace, dev, "workspace"), nbytes
    _call(_lib.moe_ep_adapter_linear, dev, a)
    _written(given)
    return out


def adapter_linear_workspace_bytes(rows: int, rank: int) -> int:
    """Bytes of workspace ``adapter_linear`` takes for these sizes."""
    a = _lib.moe_ep_adapter_args(num_rows=_int32(rows, "row count"), rank=_int32(rank, "rank"), num_adapters=1,
                                 in_features=8, out_features=1)
    return _lib.moe_ep_adapter_workspace_bytes(a)
