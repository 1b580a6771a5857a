"""The expert-side operators' host side on the CPU: struct layouts, argument
checks through the C ABI (nothing here launches: every call fails its checks
or has no rows), the 4-bit packing, and the reference's own pins."""

from __future__ import annotations

import ctypes
import math
import os
import subprocess

import pytest
import torch

from combine_token_dest_amd import W4Weights, _lib
from tests import experts_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40               # a 256-byte aligned address that is never dereferenced

INVALID, ALIGN = _lib.MOE_EP_ERR_INVALID_ARG, _lib.MOE_EP_ERR_ALIGN


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        import combine_token_dest_amd.build as b
        b.build()
    return _lib.load()


def status(fn, *args):
    try:
        fn(*args)
    except _lib.MoeEpError as e:
        return e.status
    return _lib.MOE_EP_OK


def test_struct_layouts_and_constants(tmp_path):
    structs = {n: getattr(_lib, n) for n in ("moe_ep_router", "moe_ep_weight", "moe_ep_linear_args",
                                             "moe_ep_layer_args")}
    consts = ["MOE_EP_MAX_EXPERTS", "MOE_EP_MAX_TOPK", "MOE_EP_MAX_GROUPS", "MOE_EP_SCORE_SOFTMAX", "MOE_EP_SCORE_SIGMOID"]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_ep.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} sizeof %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines += [f'printf("const {c} %d\\n", (int){c});' for c in consts] + ["return 0; }"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    seen = 0
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, f, value = line.split()
        if name == "const":
            got = getattr(_lib, f)
        else:
            got = ctypes.sizeof(structs[name]) if f == "sizeof" else getattr(structs[name], f).offset
        assert got == int(value), line
        seen += 1
    assert seen == sum(1 + len(c._fields_) for c in structs.values()) + len(consts)


def router(**kw):
    base = dict(num_experts=16, top_k=4, score=0, num_groups=1, top_groups=1, group_top=2, renormalize=1,
                invalid_expert_id=-1, scale=1.0, bias=None)
    base.update(kw)
    return _lib.moe_ep_router(**base)


def route(r, logits=FAKE, dtype=_lib.MOE_EP_F32, stride=16, n=4, ids=FAKE, w=FAKE):
    return status(_lib.moe_ep_route, r, logits, dtype, stride, n, ids, w, None)


def test_route_refusals():
    assert route(router(), n=0) == _lib.MOE_EP_OK
    for kw in (dict(num_experts=0), dict(num_experts=1025), dict(top_k=0), dict(top_k=17),
               dict(num_experts=128, top_k=65), dict(score=2), dict(num_groups=0), dict(num_groups=3), dict(num_experts=128, num_groups=128, top_groups=64),
               dict(num_groups=4, top_groups=0), dict(num_groups=4, top_groups=5),
               dict(num_groups=8, top_groups=1, top_k=4), dict(group_top=0), dict(group_top=3)):
        assert route(router(**kw), n=0) == INVALID, kw
    assert route(router(), n=-1) == INVALID
    assert route(router(), dtype=7) == INVALID
    assert route(router(), stride=15) == INVALID
    assert route(router(), stride=-16) == INVALID
    assert route(router(), stride=1 << 62) == INVALID
    assert route(router(), logits=None) == INVALID
    assert route(router(), ids=None) == INVALID
    assert route(router(), w=None) == INVALID
    assert route(router(), logits=FAKE + 2) == ALIGN
    assert route(router(), logits=FAKE + 1, dtype=_lib.MOE_EP_BF16) == ALIGN
    assert route(router(), ids=FAKE + 2) == ALIGN
    assert route(router(), w=FAKE + 1) == ALIGN
    assert route(router(bias=FAKE + 2)) == ALIGN


def linear_args(**kw):
    a = _lib.moe_ep_linear_args(x=FAKE, x_stride=64, expert_ids=FAKE, out=2 * FAKE, out_stride=32,
                                weight=_lib.moe_ep_weight(FAKE, None, 0), dtype=_lib.MOE_EP_BF16,
                                out_dtype=_lib.MOE_EP_BF16, num_rows=3, num_experts=2, expert_offset=0,
                                in_features=64, out_features=32)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def linear(**kw):
    return status(_lib.moe_ep_expert_linear, linear_args(**kw), None)


def test_linear_refusals():
    W = _lib.moe_ep_weight
    assert linear(num_rows=0) == _lib.MOE_EP_OK
    assert linear(num_rows=0, x=None, out=None) == _lib.MOE_EP_OK
    for kw in (dict(dtype=_lib.MOE_EP_F32), dict(dtype=9), dict(out_dtype=_lib.MOE_EP_F16), dict(num_rows=-1),
               dict(num_experts=0), dict(num_experts=1025), dict(expert_offset=-1), dict(expert_offset=2 ** 31 - 2),
               dict(in_features=0), dict(in_features=7), dict(out_features=0), dict(in_features=(1 << 24) + 1), dict(x=None),
               dict(out=None), dict(x_stride=63), dict(x_stride=-1), dict(out_stride=31), dict(out_stride=0),
               dict(x_stride=1 << 62), dict(weight=W(None, None, 0)), dict(weight=W(FAKE, None, 32)),
               dict(weight=W(FAKE, FAKE, 16)), dict(weight=W(FAKE, FAKE, -32)),
               dict(out=FAKE), dict(out=FAKE + 2 * 64 * 2 + 126)):
        assert linear(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 1), dict(out=2 * FAKE + 1), dict(expert_ids=FAKE + 2), dict(weight=W(FAKE + 1, None, 0)),
               dict(weight=W(FAKE + 8, FAKE, 32)), dict(weight=W(FAKE, FAKE + 8, 32)),
               dict(out=2 * FAKE + 2, out_dtype=_lib.MOE_EP_F32)):
        assert linear(**kw) == ALIGN, kw


def layer_args(**kw):
    W = _lib.moe_ep_weight
    a = _lib.moe_ep_layer_args(hidden=FAKE, hidden_stride=64, topk_ids=FAKE, topk_weights=FAKE, out=2 * FAKE,
                               out_stride=64, gate_up=W(FAKE, None, 0), down=W(FAKE, None, 0), workspace=3 * FAKE,
                               workspace_bytes=1 << 20, dtype=_lib.MOE_EP_BF16, out_dtype=_lib.MOE_EP_BF16,
                               num_tokens=3, top_k=2, num_experts=4, expert_offset=0, hidden_size=64,
                               intermediate_size=32)
    for k, v in kw.items():
        setattr(a, k, ctypes.pointer(v) if k == "router" and v is not None else v)
    return a


def layer(**kw):
    return status(_lib.moe_ep_layer, layer_args(**kw), None)


def test_layer_refusals():
    W = _lib.moe_ep_weight
    assert layer(num_tokens=0) == _lib.MOE_EP_OK
    assert layer(num_tokens=0, workspace=None, hidden=None, out=None, topk_ids=None) == _lib.MOE_EP_OK
    r = dict(router=router(num_experts=16, top_k=2), topk_ids=None, topk_weights=None, router_logits=FAKE,
             logits_stride=16, logits_dtype=_lib.MOE_EP_F32)
    assert layer(**dict(r, num_tokens=0)) == _lib.MOE_EP_OK
    for kw in (dict(dtype=_lib.MOE_EP_F32), dict(out_dtype=_lib.MOE_EP_F16), dict(num_tokens=-1), dict(top_k=0),
               dict(top_k=65), dict(num_experts=0), dict(num_experts=1025), dict(expert_offset=-1),
               dict(hidden_size=7), dict(intermediate_size=7), dict(hidden=None), dict(out=None),
               dict(topk_ids=None), dict(hidden_stride=63), dict(out_stride=63), dict(out_stride=0),
               dict(gate_up=W(None, None, 0)), dict(down=W(FAKE, None, 64)), dict(down=W(FAKE, FAKE, 48)),
               dict(workspace=None), dict(workspace_bytes=100), dict(out=FAKE + 64), dict(out=FAKE, out_stride=128),
               dict(out=FAKE, out_dtype=_lib.MOE_EP_F32), dict(r, topk_ids=FAKE), dict(r, topk_weights=FAKE),
               dict(r, top_k=3), dict(r, router_logits=None), dict(r, logits_stride=8),
               dict(r, router=router(num_experts=16, top_k=2, score=5))):
        assert layer(**kw) == INVALID, kw
    for kw in (dict(hidden=FAKE + 1), dict(out=2 * FAKE + 1), dict(topk_ids=FAKE + 2), dict(topk_weights=FAKE + 2),
               dict(workspace=3 * FAKE + 128), dict(gate_up=W(FAKE + 1, None, 0)), dict(r, router_logits=FAKE + 2)):
        assert layer(**kw) == ALIGN, kw


def test_sides_a_launch_can_cover():
    side = 1 << 22
    for kw in (dict(hidden_size=side + 1), dict(intermediate_size=side + 1)):
        assert layer(**dict(kw, num_tokens=0)) == INVALID
    assert layer(num_tokens=0, hidden_size=side, hidden_stride=side, out_stride=side) == _lib.MOE_EP_OK
    assert linear(num_rows=0, out_features=side + 1, out_stride=side + 1) == INVALID
    assert linear(num_rows=0, out_features=side, out_stride=side) == _lib.MOE_EP_OK


def test_layer_workspace_bytes():
    def size(**kw):
        return _lib.moe_ep_layer_workspace_bytes(layer_args(**kw))

    n, k, inter = 5, 3, 40
    assert size(num_tokens=0) >= 256
    got = size(num_tokens=n, top_k=k, num_experts=64, intermediate_size=inter)
    assert got >= 2 * n * k * 48 * 2 and got % 256 == 0
    assert size(num_tokens=n, top_k=k, num_experts=64, intermediate_size=inter, router=router()) > got
    # it does not grow past one pass
    assert size(num_tokens=2048, num_experts=8) == size(num_tokens=10 ** 6, num_experts=8)
    for kw in (dict(num_tokens=-1), dict(top_k=0), dict(num_experts=0), dict(intermediate_size=0)):
        assert status(_lib.moe_ep_layer_workspace_bytes, layer_args(**kw)) == INVALID


@pytest.mark.parametrize("g", [0, 32])
@pytest.mark.parametrize("E,k,H,I", [(1, 1, 64, 32), (8, 2, 4096, 1408), (32, 8, 1024, 512), (256, 8, 200, 40),
                                     (16, 8, 7168, 2048), (1024, 64, 8, 8)])
def test_layer_workspace_grows_with_the_tokens(E, k, H, I, g):
    last = 0
    for n in list(range(0, 130)) + [200, 256, 300, 512, 700, 1024, 1500, 2047, 2048, 2049, 100000]:
        a = layer_args(num_tokens=n, num_experts=E, top_k=k, hidden_size=H, intermediate_size=I)
        a.gate_up.group_size = g
        size = _lib.moe_ep_layer_workspace_bytes(a)
        assert size >= last, n
        last = size


def formula_tiles(q, s, g):
    """data and scales written from the header's formula, one element at a time."""
    E, N, K = q.shape
    nt, kb = -(-N // 16), -(-K // 128)
    data = torch.full((E, nt, kb, 1024), 0x88, dtype=torch.uint8)
    sc = torch.zeros((E, nt, kb * 128 // g, 16), dtype=s.dtype)
    for e in range(E):
        for n in range(N):
            for k in range(K):
                r, c = n % 16, k % 128
                j, i, el = c // 32, c % 32 // 8, c % 8
                at = (16 * i + r) * 16 + 4 * j + el % 4
                old = int(data[e, n // 16, k // 128, at])
                v = int(q[e, n, k])
                data[e, n // 16, k // 128, at] = (old & 0xF0) | v if el < 4 else (old & 0x0F) | v << 4
                sc[e, n // 16, k // g, r] = s[e, n, k // g]
    return data, sc


@pytest.mark.parametrize("E,N,K,g", [(1, 16, 128, 32), (2, 19, 150, 64), (1, 3, 300, 128), (1, 17, 40, 32)])
def test_pack_follows_the_header(E, N, K, g):
    gen = torch.Generator().manual_seed(K)
    q = torch.randint(0, 16, (E, N, K), generator=gen, dtype=torch.uint8)
    s = torch.randn(E, N, -(-K // g), generator=gen).to(torch.bfloat16)
    w = W4Weights.pack(q, s)
    data, sc = formula_tiles(q, s, g)
    assert w.group_size == g and torch.equal(w.data, data) and torch.equal(w.scales, sc)
    q2, s2 = w.unpack()
    assert torch.equal(q2, q) and torch.equal(s2, s)
    want, _ = ref.W4(q, s, g).expert(0)
    assert torch.equal(w.dequantize()[0].double(), want)      # 4-bit times 8-bit: exact in float32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("g,K", [(32, 96), (64, 100), (128, 40), (128, 256)])
def test_quantize(dtype, g, K):
    """Off by at most half a scale step, plus the scale's own rounding (7 steps of it)."""
    w = torch.randn(2, 20, K, generator=torch.Generator().manual_seed(g)).to(dtype)
    w[0, 3] = 0
    p = W4Weights.quantize(w, g)
    assert p.rows == 20 and p.cols == K and p.scales.dtype == dtype
    for k0 in range(0, K, g):
        part = w[:, :, k0:k0 + g].double()
        top = part.abs().amax(2, keepdim=True)
        err = (p.dequantize()[:, :, k0:k0 + g].double() - part).abs()
        assert (err <= top / 7 * (0.5 + 8 * ref.HALF_STEP[dtype])).all()
    assert torch.equal(W4Weights.quantize(w[0], g).data, p.data[:1])


def test_pack_and_quantize_refusals():
    q = torch.zeros(1, 16, 128, dtype=torch.uint8)
    for bad in (lambda: W4Weights.pack(q[0], torch.ones(1, 16, 1).half()),
                lambda: W4Weights.pack(q, torch.ones(1, 16, 3).half()),
                lambda: W4Weights.pack(q, torch.ones(1, 16, 1)),
                lambda: W4Weights.quantize(torch.ones(16, 128)),
                lambda: W4Weights.quantize(torch.ones(16, 128).half(), 48)):
        with pytest.raises((ValueError, TypeError)):
            bad()


def test_reference_route_pins():
    """The reference on hand-worked cases."""
    x = torch.tensor([[0.0, math.log(3.0), -math.inf, 0.0]])
    ids, w = ref.route(x, 3, renormalize=False)
    assert ids == [[1, 0, 3]] and w[0] == pytest.approx([0.6, 0.2, 0.2])
    ids, w = ref.route(x, 4)
    assert ids == [[1, 0, 3, -1]] and w[0] == pytest.approx([0.6, 0.2, 0.2, 0.0])
    # the bias chooses, the score weighs
    ids, w = ref.route(torch.zeros(1, 4), 2, score="sigmoid", bias=torch.tensor([0.0, 1.0, 0.5, -1.0]), scale=3.0)
    assert ids == [[1, 2]] and w[0] == pytest.approx([1.5, 1.5])
    # two groups of two: the second has the larger sum, the first the largest member
    x = torch.tensor([[2.0, -9.0, 1.0, 1.0]])
    assert ref.route(x, 1, score="sigmoid", num_groups=2, top_groups=1)[0] == [[2]]
    assert ref.route(x, 1, score="sigmoid", num_groups=2, top_groups=1, group_top=1)[0] == [[0]]
