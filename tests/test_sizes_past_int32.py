"""Sizes that the library's 32-bit arguments do not hold are refused by the
torch wrappers, not wrapped to what is left of them.  The tensors are of the
meta device, which has sizes and no memory; the library is never reached."""

from __future__ import annotations

import pytest
import torch

from combine_token_dest_amd import (adapter_linear, adapter_linear_workspace_bytes, dense, expert_linear, experts,
                                    gated_linear, moe_layer, moe_layer_workspace_bytes, rms_norm)

BIG = 2 ** 32 + 16           # wrapped to 16


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def reached(*_):
        raise AssertionError("the library was called")
    for module in (dense, experts):
        monkeypatch.setattr(module, "_activations", lambda x, what: x.get_device())
        monkeypatch.setattr(module, "_call", reached)


def adapter(n=1, N=8, K=8, L=2, R=1):
    return lambda: adapter_linear(meta(n, K), meta(N, K), meta(L, R, K), meta(L, N, R), meta(n, dtype=torch.int32),
                                  workspace=meta(256, dtype=torch.uint8))


def layer(n=1, E=2, k=2, H=8, inter=8):
    return lambda: moe_layer(meta(n, H), meta(E, 2 * inter, H), meta(E, H, inter), meta(n, k, dtype=torch.int32),
                             workspace=meta(256, dtype=torch.uint8))


@pytest.mark.parametrize("call,what", [
    (adapter(n=BIG), "row count"), (adapter(N=BIG), "out_features"), (adapter(K=BIG), "in_features"),
    (adapter(L=BIG), "adapter count"), (adapter(R=BIG), "rank"),
    (lambda: gated_linear(meta(BIG, 8), meta(16, 8)), "row count"),
    (lambda: gated_linear(meta(1, 8), meta(2 * BIG, 8)), "intermediate size"),
    (lambda: gated_linear(meta(1, BIG), meta(16, BIG)), "hidden size"),
    (lambda: rms_norm(meta(BIG, 8), meta(8)), "row count"), (lambda: rms_norm(meta(1, BIG), meta(BIG)), "hidden size"),
    (lambda: expert_linear(meta(BIG, 8), meta(2, 8, 8)), "row count"),
    (lambda: expert_linear(meta(1, 8), meta(BIG, 8, 8)), "expert count"),
    (lambda: expert_linear(meta(1, 8), meta(2, BIG, 8)), "out_features"),
    (lambda: expert_linear(meta(1, BIG), meta(2, 8, BIG)), "in_features"),
    (layer(n=BIG), "token count"), (layer(E=BIG), "expert count"), (layer(k=BIG), "top_k"), (layer(H=BIG), "hidden size"),
    (layer(inter=BIG), "intermediate size"),
    (lambda: adapter_linear_workspace_bytes(BIG, 16), "row count"),
    (lambda: adapter_linear_workspace_bytes(4, BIG), "rank"),
    (lambda: adapter_linear_workspace_bytes(-BIG, 16), "row count"),
    (lambda: moe_layer_workspace_bytes(BIG, 2, 8, 64, 64), "token count"),
    (lambda: moe_layer_workspace_bytes(2, BIG, 8, 64, 64), "top_k"),
    (lambda: moe_layer_workspace_bytes(2, 2, BIG, 64, 64), "expert count"),
    (lambda: moe_layer_workspace_bytes(2, 2, 8, BIG, 64), "hidden size"),
    (lambda: moe_layer_workspace_bytes(2, 2, 8, 64, BIG), "intermediate size")])
def test_refused(call, what):
    with pytest.raises(ValueError, match=what), torch.no_grad():
        call()


@pytest.mark.parametrize("call", [adapter(), layer(), lambda: gated_linear(meta(1, 8), meta(16, 8)),
                                  lambda: rms_norm(meta(1, 8), meta(8)), lambda: expert_linear(meta(1, 8), meta(2, 8, 8))])
def test_sizes_inside_reach_the_library(call):
    with pytest.raises(AssertionError, match="library"), torch.no_grad():
        call()
