"""Forward-mode derivatives on the CPU: no operator has them, so tensors that
carry a tangent are refused (a result without one would read as a derivative of
zero), under torch.no_grad() too, which does not end forward mode."""

from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

from combine_token_dest_amd import (Router, W4Weights, adapter_linear, expert_linear, gated_linear, moe_layer, rms_norm,
                                    route)

BF16 = torch.bfloat16


def zeros(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def w4(E, N, K):
    return W4Weights.quantize(torch.ones(E, N, K, dtype=BF16))


IDS = torch.zeros(2, dtype=torch.int32)
CALLS = {
    "rms_norm": (lambda t: rms_norm(t["x"], t["weight"], t["residual"]),
                 dict(x=zeros(2, 64), weight=zeros(64), residual=zeros(2, 64))),
    "gated_linear": (lambda t: gated_linear(t["x"], t["gate_up"], out=t["out"]),
                     dict(x=zeros(2, 64), gate_up=zeros(16, 64), out=zeros(2, 8))),
    "adapter_linear": (lambda t: adapter_linear(t["x"], t["weight"], t["a"], t["b"], IDS, scales=t["scales"]),
                       dict(x=zeros(2, 64), weight=zeros(8, 64), a=zeros(3, 4, 64), b=zeros(3, 8, 4),
                            scales=zeros(3, dtype=torch.float32))),
    "route": (lambda t: route(t["logits"], Router(2)), dict(logits=zeros(2, 8))),
    "expert_linear": (lambda t: expert_linear(t["x"], t["weight"], IDS), dict(x=zeros(2, 64), weight=zeros(4, 8, 64))),
    "moe_layer": (lambda t: moe_layer(t["x"], t["gate_up"], t["down"], router_logits=t["logits"], router=Router(2)),
                  dict(x=zeros(2, 64), gate_up=zeros(4, 32, 64), down=zeros(4, 64, 16), logits=zeros(2, 4))),
}


@pytest.mark.parametrize("op,which", [(op, name) for op, (_, t) in CALLS.items() for name in t])
@pytest.mark.parametrize("mode", ["grad", "no_grad"])
def test_a_tangent_is_refused(op, which, mode):
    call, tensors = CALLS[op]
    with forward_ad.dual_level():
        t = dict(tensors)
        t[which] = forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        with torch.set_grad_enabled(mode == "grad"), pytest.raises(RuntimeError, match=f"{op} has no forward-mode"):
            call(t)


def test_a_tangent_of_packed_weights_is_refused():
    w = w4(4, 16, 128)
    with forward_ad.dual_level():
        dual = W4Weights(w.data, forward_ad.make_dual(w.scales, torch.ones_like(w.scales)), w.rows, w.cols)
        with pytest.raises(RuntimeError, match="forward-mode"):
            expert_linear(zeros(2, 128), dual, IDS)


@pytest.mark.parametrize("op", list(CALLS))
def test_other_tensors_inside_a_dual_level_go_on(op):
    """Only tangents are refused: a call without any meets its other checks."""
    call, tensors = CALLS[op]
    with forward_ad.dual_level():
        forward_ad.make_dual(zeros(3), zeros(3))
        with pytest.raises(ValueError, match="GPU"):
            call(dict(tensors))


def test_jvp_is_refused():
    x, w = zeros(2, 64), zeros(16, 64)
    with pytest.raises(RuntimeError, match="forward-mode"):
        torch.func.jvp(lambda x: gated_linear(x, w), (x,), (torch.ones_like(x),))
