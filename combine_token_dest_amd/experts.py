"""The expert side of a mixture-of-experts step over torch tensors: what a
decode step computes around dispatch and combine.

* ``route``          a router's logits to each token's expert ids and weights
* ``expert_linear``  each row times its expert's matrix
* ``moe_layer``      the gated feed-forward of every token's experts, summed

Every step runs in the library's gfx950 kernels (include/moe_ep.h); torch is
used for device memory and the current stream.  Work is enqueued on the
current stream of the tensors' device; what a call needs beyond its inputs
comes from torch's allocator for that stream, so calls may be captured into
graphs and run on several streams at once.  There is no backward pass: tensors
that require gradients are refused outside ``torch.no_grad()``, and tensors that
carry a forward-mode derivative everywhere.
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Tuple, Union

import torch
from torch.autograd import forward_ad

from . import _lib
from ._lib import MOE_EP_BF16, MOE_EP_F16, MOE_EP_F32

_DTYPES = {torch.bfloat16: MOE_EP_BF16, torch.float16: MOE_EP_F16, torch.float32: MOE_EP_F32}
_SCORES = {"softmax": _lib.MOE_EP_SCORE_SOFTMAX, "sigmoid": _lib.MOE_EP_SCORE_SIGMOID}

_TILE_ROWS, _TILE_COLS, _TILE_BYTES = 16, 128, 1024


@dataclass
class Router:
    """How logits choose experts; see include/moe_ep.h, moe_ep_router.

    ``score`` is "softmax" or "sigmoid".  ``bias`` (float32 [num_experts] on
    the GPU) is added to the scores for the choice only.  With ``num_groups``
    above 1 only the ``top_groups`` groups whose ``group_top`` best choices
    sum highest stay open."""

    top_k: int
    score: str = "softmax"
    bias: Optional[torch.Tensor] = None
    num_groups: int = 1
    top_groups: int = 1
    group_top: int = 2
    renormalize: bool = True
    scale: float = 1.0
    invalid_expert_id: int = -1


@dataclass
class W4Weights:
    """4-bit matrices [num_experts, rows, cols] in the library's tiles:
    W[e, n, k] = (q - 8) * scale[e, n, k // group_size], q in 0..15.

    ``data`` uint8 [num_experts, ceil(rows/16), ceil(cols/128), 1024] and
    ``scales`` (bfloat16 or float16, the activations' type) [num_experts,
    ceil(rows/16), ceil(cols/128) * 128 / group_size, 16]; include/moe_ep.h,
    moe_ep_weight, has the order inside a tile.  ``quantize`` makes them from
    dense weights and ``pack`` from integers and scales."""

    data: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @property
    def num_experts(self) -> int:
        return self.data.shape[0]

    @property
    def group_size(self) -> int:
        return self.data.shape[2] * _TILE_COLS // max(1, self.scales.shape[2])

    @classmethod
    def pack(cls, q: torch.Tensor, scales: torch.Tensor) -> "W4Weights":
        """From integers ``q`` [experts, rows, cols] in 0..15 and ``scales``
        [experts, rows, ceil(cols / g)], g = 32, 64 or 128 (the smallest that
        this number of groups covers all columns with)."""
        if q.dim() != 3 or scales.dim() != 3 or scales.shape[:2] != q.shape[:2]:
            raise ValueError("q must be [experts, rows, cols] and scales [experts, rows, groups]")
        if scales.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("scales must be bfloat16 or float16")
        E, N, K = q.shape
        g = next((g for g in (32, 64, 128) if -(-K // g) == scales.shape[2]), None)
        if g is None:
            raise ValueError(f"{scales.shape[2]} scale groups do not cover {K} columns by 32, 64 or 128")
        whole = q == q.round() if q.is_floating_point() else True
        if not bool(((q >= 0) & (q <= 15) & whole).all()):
            raise ValueError("q must be integers in 0..15")
        nt, kb = -(-N // _TILE_ROWS), -(-K // _TILE_COLS)
        full = torch.full((E, nt * _TILE_ROWS, kb * _TILE_COLS), 8, dtype=torch.uint8, device=q.device)
        full[:, :N, :K] = q.to(torch.uint8)
        # [E, tile, row, block, j, i, half, byte]: column 32 j + 8 i + 4 half + byte
        v = full.view(E, nt, _TILE_ROWS, kb, 4, 4, 2, 4)
        data = (v[..., 0, :] | (v[..., 1, :] << 4)).permute(0, 1, 3, 5, 2, 4, 6)
        sc = torch.zeros((E, nt * _TILE_ROWS, kb * _TILE_COLS // g), dtype=scales.dtype, device=scales.device)
        sc[:, :N, :scales.shape[2]] = scales
        sc = sc.view(E, nt, _TILE_ROWS, kb * _TILE_COLS // g).transpose(2, 3)
        return cls(data.reshape(E, nt, kb, _TILE_BYTES).contiguous(), sc.contiguous(), N, K)

    @classmethod
    def quantize(cls, w: torch.Tensor, group_size: int = 128) -> "W4Weights":
        """Nearest 4-bit weights of dense ``w`` [experts, rows, cols] or
        [rows, cols] (bfloat16 or float16): a group's scale is its largest
        magnitude / 7, rounded to w's type.  A group with an infinity or NaN
        becomes NaN as a whole."""
        if w.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("weights must be bfloat16 or float16")
        if group_size not in (32, 64, 128):
            raise ValueError(f"group_size {group_size} is not 32, 64 or 128")
        w = w if w.dim() == 3 else w.unsqueeze(0)
        E, N, K = w.shape
        groups = -(-K // group_size)
        x = torch.zeros((E, N, groups * group_size), dtype=torch.float32, device=w.device)
        x[:, :, :K] = w
        x = x.view(E, N, groups, group_size)
        scales = (x.abs().amax(3) / 7).to(w.dtype)
        s = scales.float().unsqueeze(3)
        q = torch.where((s > 0) & (s < math.inf), x / s, torch.zeros_like(x)).round().clamp(-8, 7) + 8
        q = q.view(E, N, groups * group_size)[:, :, :K]
        # spelled out, since several group sizes can give this number of groups
        return cls._pack_groups(q, scales, group_size)

    @classmethod
    def _pack_groups(cls, q: torch.Tensor, scales: torch.Tensor, g: int) -> "W4Weights":
        K = q.shape[2]
        fits = next(x for x in (32, 64, 128) if -(-K // x) == scales.shape[2])
        if fits != g:
            # few columns: the same scales for smaller groups
            scales = scales.repeat_interleave(g // fits, 2)[:, :, :-(-K // fits)]
        return cls.pack(q, scales)

    def unpack(self) -> Tuple[torch.Tensor, torch.Tensor]:
        """(q uint8 [experts, rows, cols], scales [experts, rows, groups]):
        the inverse of ``pack``."""
        E, nt, kb, _ = self.data.shape
        d = self.data.view(E, nt, kb, 4, _TILE_ROWS, 4, 4)
        v = torch.stack((d & 15, d >> 4), -2)                    # [.., i, row, j, half, byte]
        q = v.permute(0, 1, 4, 2, 5, 3, 6, 7).reshape(E, nt * _TILE_ROWS, kb * _TILE_COLS)
        sc = self.scales.transpose(2, 3).reshape(E, nt * _TILE_ROWS, -1)
        return (q[:, :self.rows, :self.cols].contiguous(),
                sc[:, :self.rows, :-(-self.cols // self.group_size)].contiguous())

    def dequantize(self) -> torch.Tensor:
        """The weights as float32 [experts, rows, cols]."""
        q, sc = self.unpack()
        s = sc.float().repeat_interleave(self.group_size, 2)[:, :, :self.cols]
        return (q.float() - 8) * s


Weight = Union[torch.Tensor, W4Weights]


def _no_tangents(what: str, *tensors) -> None:
    """Refuses tensors that carry a forward-mode derivative (the result would
    have none, which reads as zero)."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if isinstance(t, W4Weights):
                t = t.scales
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise RuntimeError(f"{what} has no forward-mode derivative, but a tensor carries a tangent: "
                                   f"call it with the primal")


def _forward_only(what: str, *tensors) -> None:
    """Refuses what autograd would have to record (the result has no graph)."""
    _no_tangents(what, *tensors)
    if torch.is_grad_enabled():
        for t in tensors:
            if isinstance(t, W4Weights):
                t = t.scales
            if t is not None and t.requires_grad:
                raise RuntimeError(f"{what} has no backward pass, but a tensor requires gradients: "
                                   f"call it under torch.no_grad() or with detached tensors")


def _on(t: torch.Tensor, dev: int, what: str) -> int:
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, expected cuda:{dev}")
    return t.data_ptr()


def _rows(t: torch.Tensor, dev: int, what: str) -> Tuple[int, int]:
    """Address and row stride of a 2-d tensor whose rows are contiguous."""
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, expected cuda:{dev}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{what} must have contiguous rows")
    return t.data_ptr(), t.stride(0)


def _weight(w: Weight, dev: int, dtype: torch.dtype, what: str, out) -> Tuple[int, int, int]:
    """Fills a moe_ep_weight; returns (experts, rows, cols)."""
    if isinstance(w, W4Weights):
        data, sc = w.data, w.scales
        E, nt, kb = data.shape[0], -(-w.rows // _TILE_ROWS), -(-w.cols // _TILE_COLS)
        if data.dtype != torch.uint8 or data.shape[1:] != (nt, kb, _TILE_BYTES):
            raise ValueError(f"{what}: data must be uint8 [{E}, {nt}, {kb}, {_TILE_BYTES}]")
        g = w.group_size
        if sc.dtype != dtype:
            raise TypeError(f"{what}: scales are {sc.dtype}, the activations {dtype}")
        if g not in (32, 64, 128) or sc.shape != (E, nt, kb * _TILE_COLS // g, _TILE_ROWS):
            raise ValueError(f"{what}: scales {tuple(sc.shape)} do not fit data {tuple(data.shape)}")
        if not (data.is_contiguous() and sc.is_contiguous()):
            raise ValueError(f"{what} must be contiguous")
        out.data, out.scales, out.group_size = _on(data, dev, what), _on(sc, dev, what), g
        return E, w.rows, w.cols
    if w.dtype != dtype:
        raise TypeError(f"{what} is {w.dtype}, the activations {dtype}")
    if w.dim() != 3 or not w.is_contiguous():
        raise ValueError(f"{what} must be a contiguous [experts, rows, cols]")
    out.data, out.scales, out.group_size = _on(w, dev, what), None, 0
    return w.shape[0], w.shape[1], w.shape[2]


def _activations(x: torch.Tensor, what: str) -> int:
    if x.dim() != 2:
        raise ValueError(f"{what} must be [rows, features]")
    if x.dtype != torch.bfloat16 and x.dtype != torch.float16:
        raise TypeError(f"{what} must be bfloat16 or float16, got {x.dtype}")
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{what} is on {x.device}, expected a GPU")
    return dev


def _output(out, shape, dtype, out_dtype, x) -> torch.Tensor:
    if out is None:
        odt = x.dtype if out_dtype is None else out_dtype
        if odt != x.dtype and odt != torch.float32:
            raise TypeError(f"out_dtype must be {x.dtype} or float32, got {odt}")
        return x.new_empty(shape, dtype=odt)
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    if tuple(out.shape) != tuple(shape) or (out.dtype != dtype and out.dtype != torch.float32):
        raise ValueError(f"out must be {dtype} or float32 {list(shape)}")
    return out


def int32_ids(t: torch.Tensor) -> torch.Tensor:
    """int64 expert ids as the library's int32.  What int32 does not hold
    becomes its first or last value, which names no expert either (wrapped, it
    could)."""
    return t.clamp(-0x80000000, 0x7fffffff).to(torch.int32)


def _ids(t: torch.Tensor, shape, dev: int, what: str) -> torch.Tensor:
    if t.dtype == torch.int64:
        t = int32_ids(t)
    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be int32 (or int64, converted) {list(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, expected cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _router(r: Router, num_experts: int, dev: int) -> "_lib.moe_ep_router":
    if r.score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {r.score!r}")
    if not math.isfinite(r.scale):
        raise ValueError(f"scale must be finite, got {r.scale}")
    bias = None
    if r.bias is not None:
        b = r.bias
        if b.dtype != torch.float32 or tuple(b.shape) != (num_experts,) or not b.is_contiguous():
            raise ValueError(f"bias must be a contiguous float32 [{num_experts}]")
        bias = _on(b, dev, "bias")
    return _lib.moe_ep_router(num_experts, r.top_k, _SCORES[r.score], r.num_groups, r.top_groups, r.group_top,
                              1 if r.renormalize else 0, r.invalid_expert_id, r.scale, bias)


def _logits(logits: torch.Tensor) -> Tuple[int, int, int]:
    """(device, dtype, row stride) of router logits."""
    if logits.dim() != 2 or logits.dtype not in _DTYPES:
        raise ValueError("logits must be [tokens, experts] of float32, bfloat16 or float16")
    dev = logits.get_device()
    if dev < 0:
        raise ValueError(f"logits are on {logits.device}, expected a GPU")
    if logits.stride(1) != 1 and logits.shape[1] > 1:
        raise ValueError("logits must have contiguous rows")
    return dev, _DTYPES[logits.dtype], logits.stride(0)


def _int32(n: int, what: str) -> int:
    if n > 0x7fffffff or n < 0:
        raise ValueError(f"{what} {n} is not in [0, 2^31)")
    return n


def _call(entry, dev: int, *args) -> None:
    """entry(*args, stream) on the current stream of GPU ``dev``, with that
    device current.  (The raw accessors: torch.cuda.current_stream() builds a
    Stream object, a tenth of a call's host time.)"""
    if torch._C._cuda_getDevice() == dev:
        entry(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            entry(*args, torch._C._cuda_getCurrentRawStream(dev))


def _written(*outputs: Optional[torch.Tensor]) -> None:
    """Counts a new version of the caller's outputs, as torch's own operators
    do: a backward pass that saved one refuses what is there now."""
    for t in outputs:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def route(logits: torch.Tensor, router: Router, *, topk_ids: Optional[torch.Tensor] = None,
          topk_weights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Each token's ``top_k`` expert ids (int32) and weights (float32), both
    [tokens, top_k], from ``logits`` [tokens, experts] (float32, bfloat16 or
    float16; rows may be strided): what ``MoEEp.dispatch`` and ``moe_layer``
    take.  Ties go to the lowest id; an expert whose logit or bias is -inf or
    NaN is never chosen, and a slot left without one gets
    ``invalid_expert_id`` and weight 0.  See include/moe_ep.h, moe_ep_route."""
    _forward_only("route", logits, router.bias, topk_weights)
    dev, dtype, stride = _logits(logits)
    n, E = logits.shape
    _int32(n, "token count")
    r = _router(router, E, dev)
    shape, given = (n, router.top_k), (topk_ids, topk_weights)
    if topk_ids is None:
        topk_ids = logits.new_empty(shape, dtype=torch.int32)
    elif topk_ids.dtype != torch.int32 or tuple(topk_ids.shape) != shape or not topk_ids.is_contiguous():
        raise ValueError(f"topk_ids must be a contiguous int32 {list(shape)}")
    if topk_weights is None:
        topk_weights = logits.new_empty(shape, dtype=torch.float32)
    elif topk_weights.dtype != torch.float32 or tuple(topk_weights.shape) != shape \
            or not topk_weights.is_contiguous():
        raise ValueError(f"topk_weights must be a contiguous float32 {list(shape)}")
    _call(_lib.moe_ep_route, dev, r, logits.data_ptr(), dtype, stride, n, _on(topk_ids, dev, "topk_ids"),
          _on(topk_weights, dev, "topk_weights"))
    _written(*given)
    return topk_ids, topk_weights


def expert_linear(x: torch.Tensor, weight: Weight, expert_ids: Optional[torch.Tensor] = None, *,
                  expert_offset: int = 0, out: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """``out[r] = weight[expert_ids[r] - expert_offset] @ x[r]``.

    ``x`` [rows, in] is bfloat16 or float16 (rows may be strided), ``weight``
    a dense [experts, out, in] of its type or a ``W4Weights``.  Rows whose id
    is outside [expert_offset, expert_offset + experts) get zeros; without
    ``expert_ids`` every row is multiplied with the first expert's matrix.
    The result is of x's type or float32 (``out_dtype``).  Made for the few
    rows of a decode step; see include/moe_ep.h, moe_ep_expert_linear."""
    _forward_only("expert_linear", x, weight, out)
    dev = _activations(x, "x")
    a = _lib.moe_ep_linear_args()
    E, N, K = _weight(weight, dev, x.dtype, "weight", a.weight)
    n = x.shape[0]
    if x.shape[1] != K:
        raise ValueError(f"x has {x.shape[1]} features, weight {K}")
    given, out = out, _output(out, (n, N), x.dtype, out_dtype, x)
    a.x, a.x_stride = _rows(x, dev, "x")
    a.out, a.out_stride = _rows(out, dev, "out")
    if expert_ids is not None:
        expert_ids = _ids(expert_ids, (n,), dev, "expert_ids")
        a.expert_ids = expert_ids.data_ptr()
    a.dtype, a.out_dtype = _DTYPES[x.dtype], _DTYPES[out.dtype]
    a.num_rows, a.num_experts = _int32(n, "row count"), _int32(E, "expert count")
    a.expert_offset = _int32(expert_offset, "expert_offset")
    a.in_features, a.out_features = _int32(K, "in_features"), _int32(N, "out_features")
    _call(_lib.moe_ep_expert_linear, dev, a)
    _written(given)
    return out


def moe_layer(hidden: torch.Tensor, gate_up: Weight, down: Weight, topk_ids: Optional[torch.Tensor] = None,
              topk_weights: Optional[torch.Tensor] = None, *, router_logits: Optional[torch.Tensor] = None,
              router: Optional[Router] = None, expert_offset: int = 0, out: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``out[t] = sum_j w[t, j] * down_e(silu(gate_e(x_t)) * up_e(x_t))`` over
    the experts e = ids[t, j] - expert_offset whose weights are here.

    ``hidden`` [tokens, hidden] is bfloat16 or float16; ``gate_up`` [experts,
    2 * intermediate, hidden] holds the gate rows, then the up rows, ``down``
    [experts, hidden, intermediate]; each is dense of hidden's type or a
    ``W4Weights``.  Ids and weights come from ``topk_ids`` (int32 or int64)
    and ``topk_weights`` (float32; None: all 1), [tokens, top_k], or are
    chosen from ``router_logits`` by ``router``.  Ids of other experts are
    skipped, and a token with none gets zeros, so the rows and ids that
    dispatch left a rank can be passed as they are.

    ``workspace`` (uint8, ``moe_layer_workspace_bytes`` of it) is taken from
    torch's allocator when not passed; one that is passed must not be used by
    two calls that may overlap in time.  See include/moe_ep.h, moe_ep_layer."""
    _forward_only("moe_layer", hidden, gate_up, down, topk_weights, router_logits,
                  None if router is None else router.bias, out)
    dev = _activations(hidden, "hidden")
    a = _lib.moe_ep_layer_args()
    dtype = hidden.dtype
    E, N, H = _weight(gate_up, dev, dtype, "gate_up", a.gate_up)
    E2, H2, inter = _weight(down, dev, dtype, "down", a.down)
    if E != E2 or N != 2 * inter or H != H2:
        raise ValueError(f"gate_up [{E}, {N}, {H}] and down [{E2}, {H2}, {inter}] do not belong together")
    n = hidden.shape[0]
    if hidden.shape[1] != H:
        raise ValueError(f"hidden has {hidden.shape[1]} features, gate_up {H}")
    if router is not None:
        if topk_ids is not None or topk_weights is not None or router_logits is None:
            raise ValueError("pass topk_ids (and topk_weights), or router_logits and router")
        ldev, a.logits_dtype, a.logits_stride = _logits(router_logits)
        if router_logits.shape[0] != n or ldev != dev:
            raise ValueError(f"router_logits must be [{n}, experts] on cuda:{dev}")
        r = _router(router, router_logits.shape[1], dev)
        a.router = ctypes.pointer(r)
        a.router_logits = router_logits.data_ptr()
        top_k = router.top_k
    else:
        if topk_ids is None or router_logits is not None:
            raise ValueError("pass topk_ids (and topk_weights), or router_logits and router")
        top_k = topk_ids.shape[1] if topk_ids.dim() == 2 else 0
        topk_ids = _ids(topk_ids, (n, top_k), dev, "topk_ids")
        a.topk_ids = topk_ids.data_ptr()
        if topk_weights is not None:
            w = topk_weights
            if w.dtype != torch.float32 or tuple(w.shape) != (n, top_k) or not w.is_contiguous():
                raise ValueError(f"topk_weights must be a contiguous float32 [{n}, {top_k}]")
            a.topk_weights = _on(w, dev, "topk_weights")
    given, out = out, _output(out, (n, H), dtype, out_dtype, hidden)
    a.hidden, a.hidden_stride = _rows(hidden, dev, "hidden")
    a.out, a.out_stride = _rows(out, dev, "out")
    a.dtype, a.out_dtype = _DTYPES[dtype], _DTYPES[out.dtype]
    a.num_tokens, a.top_k, a.num_experts = _int32(n, "token count"), _int32(top_k, "top_k"), _int32(E, "expert count")
    a.expert_offset = _int32(expert_offset, "expert_offset")
    a.hidden_size, a.intermediate_size = _int32(H, "hidden size"), _int32(inter, "intermediate size")
    if workspace is None:
        nbytes = _lib.moe_ep_layer_workspace_bytes(a)
        workspace = hidden.new_empty((nbytes,), dtype=torch.uint8)
    else:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        nbytes = workspace.numel()
    a.workspace, a.workspace_bytes = _on(workspace, dev, "workspace"), nbytes
    _call(_lib.moe_ep_layer, dev, a)
    _written(given)
    return out


def moe_layer_workspace_bytes(tokens: int, top_k: int, num_experts: int, hidden: int, intermediate: int, *,
                              group_size: int = 0, routed: bool = False) -> int:
    """Bytes of workspace ``moe_layer`` takes for these sizes; ``group_size``
    is that of a 4-bit ``gate_up`` (0: dense), ``routed`` when it is given
    router logits."""
    a = _lib.moe_ep_layer_args()
    a.num_tokens, a.top_k = _int32(tokens, "token count"), _int32(top_k, "top_k")
    a.num_experts, a.gate_up.group_size = _int32(num_experts, "expert count"), group_size
    a.hidden_size, a.intermediate_size = _int32(hidden, "hidden size"), _int32(intermediate, "intermediate size")
    if routed:
        a.router = ctypes.pointer(_lib.moe_ep_router())
    return _lib.moe_ep_layer_workspace_bytes(a)
