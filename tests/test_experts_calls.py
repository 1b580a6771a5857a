"""Calls of the expert-side operators that the wrapper refuses before it looks
at devices: on the CPU, nothing is launched."""

from __future__ import annotations

import pytest
import torch

from combine_token_dest_amd import Router, W4Weights, expert_linear, moe_layer, route


def bf16(*shape, grad=False):
    return torch.zeros(*shape, dtype=torch.bfloat16).requires_grad_(grad)


@pytest.mark.parametrize("which", ["x", "weight", "scales", "out"])
def test_linear_refuses_tensors_that_require_gradients(which):
    """There is no backward pass: a result without a graph would cut the
    gradient silently."""
    x, out = bf16(2, 128, grad=which == "x"), bf16(2, 16, grad=which == "out")
    w = bf16(1, 16, 128, grad=which == "weight")
    if which == "scales":
        w = W4Weights.pack(torch.full((1, 16, 128), 8, dtype=torch.uint8), bf16(1, 16, 1))
        w.scales.requires_grad_()
    with pytest.raises(RuntimeError, match="backward"):
        expert_linear(x, w, out=out)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):      # past that check
        expert_linear(x, w, out=out)


@pytest.mark.parametrize("which", ["hidden", "gate_up", "down", "topk_weights", "router_logits", "bias", "out"])
def test_layer_refuses_tensors_that_require_gradients(which):
    def grad(t, name):
        return t.requires_grad_(which == name)

    args = (grad(bf16(2, 64), "hidden"), grad(bf16(4, 32, 64), "gate_up"), grad(bf16(4, 64, 16), "down"))
    out = grad(bf16(2, 64), "out")
    if which in ("router_logits", "bias"):
        kw = dict(router_logits=grad(torch.zeros(2, 4), "router_logits"),
                  router=Router(2, bias=grad(torch.zeros(4), "bias")))
    else:
        kw = dict(topk_ids=torch.zeros(2, 2, dtype=torch.int32),
                  topk_weights=grad(torch.zeros(2, 2), "topk_weights"))
    with pytest.raises(RuntimeError, match="backward"):
        moe_layer(*args, out=out, **kw)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        moe_layer(*args, out=out, **kw)


@pytest.mark.parametrize("which", ["logits", "bias", "topk_weights"])
def test_route_refuses_tensors_that_require_gradients(which):
    logits = torch.zeros(2, 4).requires_grad_(which == "logits")
    r = Router(2, bias=torch.zeros(4).requires_grad_(which == "bias"))
    w = torch.zeros(2, 2).requires_grad_(which == "topk_weights")
    with pytest.raises(RuntimeError, match="backward"):
        route(logits, r, topk_weights=w)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        route(logits, r, topk_weights=w)


@pytest.mark.parametrize("q", [16, -1, 255, 2.5, float("nan")])
def test_pack_refuses_what_four_bits_do_not_hold(q):
    """One such value would change its neighbour in the byte."""
    t = torch.full((1, 16, 128), 8.0)
    t[0, 3, 5] = q
    t = t if isinstance(q, float) else t.to(torch.int32)
    with pytest.raises(ValueError, match="0..15"):
        W4Weights.pack(t, torch.ones(1, 16, 1).half())


def test_pack_takes_integers_of_any_type():
    q = torch.randint(0, 16, (2, 16, 128), generator=torch.Generator().manual_seed(1), dtype=torch.uint8)
    s = torch.ones(2, 16, 4).half()
    want = W4Weights.pack(q, s).data
    for t in (q.to(torch.int8), q.long(), q.float()):
        assert torch.equal(W4Weights.pack(t, s).data, want)
    empty = W4Weights.pack(q[:0], s[:0])
    assert empty.num_experts == 0


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_marks_a_group_it_cannot_scale(dtype, bad):
    """A group with an infinity or NaN becomes NaN as a whole, not finite
    values or an infinity of the other sign; its neighbours stay."""
    w = torch.randn(1, 16, 128, generator=torch.Generator().manual_seed(2)).to(dtype)
    clean = W4Weights.quantize(w, 32).dequantize()
    w[0, 3, 40] = bad
    got = W4Weights.quantize(w, 32).dequantize()
    assert got[0, 3, 32:64].isnan().all()
    got[0, 3, 32:64] = clean[0, 3, 32:64]
    assert torch.equal(got, clean)
