"""Outputs of the caller's that the torch wrappers write into count a new
version, as torch's own operators do, so that a backward pass that saved one of
them does not go on with what is there now.  On the CPU the tensors are of the
meta device, which has versions and no memory, and the library is not reached."""

from __future__ import annotations

import pytest
import torch

from combine_token_dest_amd import (Router, adapter_linear, dense, expert_linear, experts, gated_linear, moe_layer,
                                    rms_norm, route)

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def meta(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def ids(*shape):
    return meta(*shape, dtype=torch.int32)


CALLS = {
    "norm": (lambda o: rms_norm(meta(4, 64), meta(64), meta(4, 64), **o), dict(out=meta(4, 64), residual_out=meta(4, 64))),
    "norm8": (lambda o: rms_norm(meta(4, 64), meta(64), meta(4, 64), out_dtype=E4M3, group_size=32, **o),
              dict(out=meta(4, 64, dtype=E4M3), scales=meta(4, 2, dtype=torch.float32), residual_out=meta(4, 64))),
    "gated": (lambda o: gated_linear(meta(4, 64), meta(32, 64), **o), dict(out=meta(4, 16))),
    "adapter": (lambda o: adapter_linear(meta(4, 64), meta(16, 64), meta(2, 8, 64), meta(2, 16, 8), ids(4),
                                         workspace=meta(256, dtype=torch.uint8), **o), dict(out=meta(4, 16))),
    "expert": (lambda o: expert_linear(meta(4, 64), meta(2, 16, 64), ids(4), **o), dict(out=meta(4, 16))),
    "layer": (lambda o: moe_layer(meta(4, 64), meta(2, 32, 64), meta(2, 64, 16), ids(4, 2),
                                  workspace=meta(256, dtype=torch.uint8), **o), dict(out=meta(4, 64))),
    "route": (lambda o: route(meta(4, 8), Router(2), **o),
              dict(topk_ids=ids(4, 2), topk_weights=meta(4, 2, dtype=torch.float32))),
}


@pytest.fixture
def no_library(monkeypatch):
    for module in (dense, experts):
        monkeypatch.setattr(module, "_activations", lambda x, what: x.get_device())
        monkeypatch.setattr(module, "_call", lambda *_: None)
    monkeypatch.setattr(experts, "_logits", lambda t: (t.get_device(), 1, t.stride(0)))


@pytest.mark.parametrize("op", list(CALLS))
def test_every_output_of_the_callers(op, no_library):
    call, outputs = CALLS[op]
    for given in ([n] for n in outputs):
        some = {n: outputs[n] for n in given}
        before = {n: t._version for n, t in outputs.items()}
        call(some)
        assert {n: t._version - before[n] for n, t in outputs.items()} == {n: int(n in some) for n in outputs}
    call({})


@pytest.mark.parametrize("op", list(CALLS))
def test_outputs_made_in_inference_mode(op, no_library):
    """They have no versions."""
    call, outputs = CALLS[op]
    with torch.inference_mode():
        call({n: torch.empty_like(t) for n, t in outputs.items()})


@pytest.mark.gpu
def test_a_backward_pass_notices():
    """Rows that gated_linear saved, then the next norm's in their place."""
    x, w, norm = torch.randn(6, 64).to(BF16).cuda(), torch.randn(32, 64).to(BF16).cuda(), torch.ones(64).cuda()
    w.requires_grad_()
    h = gated_linear(x, w)
    rms_norm(x, norm, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(h, w, torch.ones_like(h))
    h = gated_linear(x, w)
    rms_norm(x, norm, torch.zeros_like(x), residual_out=torch.empty_like(x))
    torch.autograd.grad(h, w, torch.ones_like(h))
