"""The dense operators' host side on the CPU: struct layouts and argument
checks through the C ABI (nothing here launches: every call fails its checks
or has no rows), and the calls the torch wrappers refuse."""

from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

from combine_token_dest_amd import _lib, adapter_linear, gated_linear, rms_norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40               # a 256-byte aligned address that is never dereferenced
INVALID, ALIGN, OK = _lib.MOE_EP_ERR_INVALID_ARG, _lib.MOE_EP_ERR_ALIGN, _lib.MOE_EP_OK
NAN, INF = float("nan"), float("inf")


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
    return OK


def bf16(*shape, grad=False, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).requires_grad_(grad)


def check_layout(tmp_path, names):
    structs = {n: getattr(_lib, n) for n in names}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_ep.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} sizeof %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines += ['printf("E4M3 const %d\\n", MOE_EP_E4M3);', "return 0; }"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, f, value = line.split()
        if f == "const":
            got = _lib.MOE_EP_E4M3
        else:
            got = ctypes.sizeof(structs[name]) if f == "sizeof" else getattr(structs[name], f).offset
        assert got == int(value), line


def test_norm_layout(tmp_path):
    check_layout(tmp_path, ["moe_ep_norm_args"])


def norm(**kw):
    base = dict(x=FAKE, x_stride=256, residual=2 * FAKE, residual_stride=256, weight=3 * FAKE, out=4 * FAKE,
                out_stride=256, scales=5 * FAKE, scales_stride=2, residual_out=6 * FAKE, residual_out_stride=256,
                dtype=_lib.MOE_EP_BF16, weight_dtype=_lib.MOE_EP_F32, out_dtype=_lib.MOE_EP_E4M3, group_size=128,
                num_rows=4, hidden_size=256, eps=1e-6)
    base.update(kw)
    return status(_lib.moe_ep_rms_norm, _lib.moe_ep_norm_args(**base), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=0), dict(dtype=8), dict(weight_dtype=2), dict(out_dtype=2), dict(out_dtype=0), dict(group_size=16),
    dict(group_size=-128), dict(out_dtype=1, scales=None), dict(out_dtype=1, group_size=0), dict(num_rows=-1),
    dict(hidden_size=7), dict(hidden_size=(1 << 22) + 1), dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF),
    dict(x_stride=255), dict(x_stride=-256), dict(x_stride=1 << 62), dict(residual_stride=255), dict(out_stride=255),
    dict(out_stride=0), dict(residual_out_stride=0), dict(scales_stride=1), dict(scales_stride=0), dict(x=None),
    dict(out=None), dict(scales=None), dict(weight=None), dict(residual=None), dict(residual=None, residual_out=6 * FAKE),
    # overlaps
    dict(out=FAKE), dict(out=FAKE + 100), dict(residual_out=FAKE + 2), dict(residual_out=2 * FAKE + 2),
    dict(residual_out=2 * FAKE, residual_out_stride=512), dict(out=6 * FAKE), dict(scales=FAKE), dict(scales=4 * FAKE),
    dict(scales=6 * FAKE), dict(out=3 * FAKE), dict(residual_out=3 * FAKE + 512), dict(scales=3 * FAKE),
    dict(out_dtype=1, group_size=0, scales=None, out=FAKE + 2),
    dict(out_dtype=1, group_size=0, scales=None, out=FAKE, out_stride=257),
    dict(out_dtype=1, group_size=0, scales=None, out=2 * FAKE, residual_out=2 * FAKE),
])
def test_norm_refusals(kw):
    assert norm(**kw) == INVALID


def test_norm_alignment():
    for kw in (dict(x=FAKE + 1), dict(residual=FAKE + 1), dict(weight=FAKE + 2), dict(residual_out=6 * FAKE + 1),
               dict(scales=5 * FAKE + 2), dict(out_dtype=1, group_size=0, scales=None, out=4 * FAKE + 1)):
        assert norm(**kw) == ALIGN, kw
    assert _lib.load().moe_ep_rms_norm(None, None) == INVALID


def test_norm_without_rows():
    assert norm(num_rows=0) == OK
    assert norm(num_rows=0, x=None, out=None, scales=None, residual=None, residual_out=None) == OK
    assert norm(num_rows=0, eps=NAN) == INVALID


@pytest.mark.parametrize("which", ["x", "weight", "residual", "out", "scales", "residual_out"])
def test_norm_refuses_tensors_that_require_gradients(which):
    t = dict(x=bf16(2, 64), weight=bf16(64), residual=bf16(2, 64), out=bf16(2, 64), scales=None,
             residual_out=bf16(2, 64))
    if which == "scales":
        t["scales"] = torch.zeros(2, 1)
    t[which].requires_grad_()
    with pytest.raises(RuntimeError, match="backward"):
        rms_norm(t.pop("x"), t.pop("weight"), **t)


def test_norm_wrapper_refusals():
    x, w = bf16(2, 64), bf16(64)
    with pytest.raises(ValueError, match="GPU"):
        rms_norm(x, w)
    with pytest.raises(ValueError, match="rows, features"):
        rms_norm(bf16(64), w)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        rms_norm(torch.zeros(2, 64), w)


def gated(**kw):
    base = dict(x=FAKE, x_stride=64, gate_up=2 * FAKE, gate_up_stride=64, out=3 * FAKE, out_stride=32, pre=4 * FAKE,
                dtype=_lib.MOE_EP_BF16, out_dtype=_lib.MOE_EP_BF16, num_rows=4, hidden_size=64, intermediate_size=32)
    base.update(kw)
    return status(_lib.moe_ep_gated, _lib.moe_ep_gated_args(**base), None)


def grad_args(**kw):
    base = dict(dout=FAKE, dout_stride=32, x=2 * FAKE, x_stride=64, gate_up=3 * FAKE, gate_up_stride=64, pre=4 * FAKE,
                dx=5 * FAKE, dx_stride=64, dgate_up=6 * FAKE, dgate_up_stride=64, workspace=7 * FAKE,
                workspace_bytes=1 << 24, dtype=_lib.MOE_EP_F16, dout_dtype=_lib.MOE_EP_F16, num_rows=4, hidden_size=64,
                intermediate_size=32)
    base.update(kw)
    return _lib.moe_ep_gated_grad_args(**base)


def grad(**kw):
    return status(_lib.moe_ep_gated_grad, grad_args(**kw), None)


def adapter_args(**kw):
    base = dict(x=FAKE, x_stride=64, weight=2 * FAKE, weight_stride=64, lora_a=3 * FAKE, lora_b=4 * FAKE,
                adapter_ids=5 * FAKE, scales=6 * FAKE, out=7 * FAKE, out_stride=32, workspace=8 * FAKE,
                workspace_bytes=4096, dtype=_lib.MOE_EP_BF16, out_dtype=_lib.MOE_EP_F32, num_rows=4, in_features=64,
                out_features=32, num_adapters=3, rank=16)
    base.update(kw)
    return _lib.moe_ep_adapter_args(**base)


def adapter(**kw):
    return status(_lib.moe_ep_adapter_linear, adapter_args(**kw), None)


def test_layouts(tmp_path):
    check_layout(tmp_path, ["moe_ep_gated_args", "moe_ep_gated_grad_args", "moe_ep_adapter_args"])


SIDE = (1 << 22) + 1


@pytest.mark.parametrize("kw", [
    dict(dtype=0), dict(out_dtype=2), dict(out_dtype=8), dict(num_rows=-1), dict(hidden_size=7), dict(hidden_size=SIDE),
    dict(intermediate_size=7), dict(intermediate_size=SIDE), dict(x_stride=63), dict(x_stride=-64), dict(x=None),
    dict(gate_up=None), dict(gate_up_stride=63), dict(gate_up_stride=0), dict(out=None), dict(out_stride=31),
    dict(out=FAKE), dict(out=2 * FAKE + 100), dict(pre=FAKE), dict(pre=3 * FAKE), dict(x_stride=1 << 62),
    dict(num_rows=2 ** 31 - 1, hidden_size=1 << 22, x_stride=1 << 22, gate_up_stride=1 << 22,
         intermediate_size=1 << 22, out_stride=1 << 22)])
def test_gated_refusals(kw):
    assert gated(**kw) == INVALID


def test_gated_alignment_and_no_rows():
    for kw in (dict(x=FAKE + 1), dict(gate_up=2 * FAKE + 1), dict(out=3 * FAKE + 1),
               dict(out=3 * FAKE + 2, out_dtype=_lib.MOE_EP_F32), dict(pre=4 * FAKE + 2)):
        assert gated(**kw) == ALIGN, kw
    assert gated(num_rows=0, x=None, out=None, pre=None) == OK
    assert gated(num_rows=0, gate_up=None) == INVALID
    assert _lib.load().moe_ep_gated(None, None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dtype=0), dict(dout_dtype=1), dict(num_rows=-1), dict(hidden_size=7), dict(intermediate_size=SIDE),
    dict(dout=None), dict(dout_stride=31), dict(x=None), dict(x_stride=63), dict(gate_up=None), dict(gate_up_stride=1),
    dict(pre=None), dict(dx_stride=63), dict(dx_stride=0), dict(dgate_up_stride=63), dict(workspace=None),
    dict(workspace_bytes=100), dict(dx=FAKE), dict(dx=6 * FAKE), dict(dgate_up=2 * FAKE), dict(dgate_up=3 * FAKE),
    dict(workspace=4 * FAKE), dict(workspace=5 * FAKE), dict(dx=4 * FAKE)])
def test_gated_grad_refusals(kw):
    assert grad(**kw) == INVALID


def test_gated_grad_alignment_and_nothing_to_do():
    for kw in (dict(dout=FAKE + 1), dict(x=2 * FAKE + 1), dict(gate_up=3 * FAKE + 1), dict(pre=4 * FAKE + 2),
               dict(dx=5 * FAKE + 1), dict(dgate_up=6 * FAKE + 1), dict(workspace=7 * FAKE + 128)):
        assert grad(**kw) == ALIGN, kw
    # no gradient asked for; without rows only dgate_up is left to write
    assert grad(dx=None, dgate_up=None, workspace=None) == OK
    assert grad(num_rows=0, dgate_up=None, workspace=None, dout=None, pre=None, dx=None) == OK
    assert _lib.load().moe_ep_gated_grad(None, None) == INVALID


def test_gated_grad_workspace():
    small = _lib.moe_ep_gated_grad_workspace_bytes(grad_args())
    assert small >= 4 * 64 * 2
    # 64-bit sizes
    a = grad_args(num_rows=2 ** 31 - 1, intermediate_size=1 << 22)
    assert _lib.moe_ep_gated_grad_workspace_bytes(a) >= (2 ** 31 - 1) * (1 << 24)
    assert status(_lib.moe_ep_gated_grad_workspace_bytes, grad_args(hidden_size=0)) == INVALID
    assert grad(workspace_bytes=small - 1) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dtype=0), dict(out_dtype=2), dict(num_rows=-1), dict(num_rows=(1 << 25) + 1, workspace_bytes=1 << 40),
    dict(num_rows=1 << 25, out_features=1 << 14, out_stride=1 << 14, workspace_bytes=1 << 40),
    dict(in_features=7), dict(in_features=SIDE),
    dict(out_features=0), dict(out_features=SIDE), dict(num_adapters=0), dict(num_adapters=1025), dict(rank=0),
    dict(rank=1025), dict(x=None), dict(x_stride=63), dict(weight=None), dict(weight_stride=63), dict(lora_a=None),
    dict(lora_b=None), dict(adapter_ids=None), dict(out=None), dict(out_stride=31), dict(workspace=None),
    dict(workspace_bytes=255), dict(out=FAKE), dict(out=2 * FAKE), dict(out=3 * FAKE + 4), dict(out=4 * FAKE),
    dict(out=5 * FAKE), dict(out=6 * FAKE), dict(out=8 * FAKE), dict(workspace=FAKE), dict(workspace=3 * FAKE)])
def test_adapter_refusals(kw):
    assert adapter(**kw) == INVALID


def test_adapter_alignment_and_no_rows():
    for kw in (dict(x=FAKE + 1), dict(weight=2 * FAKE + 1), dict(lora_a=3 * FAKE + 1), dict(lora_b=4 * FAKE + 1),
               dict(adapter_ids=5 * FAKE + 2), dict(scales=6 * FAKE + 2), dict(out=7 * FAKE + 2),
               dict(workspace=8 * FAKE + 4)):
        assert adapter(**kw) == ALIGN, kw
    assert adapter(num_rows=0, x=None, out=None, adapter_ids=None, workspace=None) == OK
    assert _lib.load().moe_ep_adapter_linear(None, None) == INVALID


@pytest.mark.parametrize("which", ["x", "gate_up", "out"])
def test_gated_refuses_out_where_autograd_records(which):
    t = dict(x=bf16(2, 64), gate_up=bf16(16, 64), out=bf16(2, 8))
    t[which].requires_grad_()
    with pytest.raises(RuntimeError, match="autograd"):
        gated_linear(t["x"], t["gate_up"], out=t["out"])
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        gated_linear(t["x"], t["gate_up"], out=t["out"])


@pytest.mark.parametrize("which", ["x", "weight", "lora_a", "lora_b", "scales", "out"])
def test_adapter_refuses_tensors_that_require_gradients(which):
    t = dict(x=bf16(2, 64), weight=bf16(8, 64), lora_a=bf16(3, 4, 64), lora_b=bf16(3, 8, 4), scales=torch.ones(3),
             out=bf16(2, 8))
    t[which].requires_grad_()
    ids = torch.zeros(2, dtype=torch.int32)
    args = (t["x"], t["weight"], t["lora_a"], t["lora_b"], ids)
    with pytest.raises(RuntimeError, match="backward"):
        adapter_linear(*args, scales=t["scales"], out=t["out"])
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        adapter_linear(*args, scales=t["scales"], out=t["out"])


def test_gated_gradient_formula_against_differences():
    """The float64 reference's gradients are those of its own h."""
    from tests import dense_ref as ref
    g = torch.Generator().manual_seed(3)
    x, w, dh = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 9), (8, 9), (3, 4)))

    def loss(x, w):
        return float((ref.gated(x, w)[2] * dh).sum())

    dx, _, dw, _ = ref.gated_grad(x, w, dh, torch.float16)
    for t, d, at in ((x, dx, lambda v: loss(v, w)), (w, dw, lambda v: loss(x, v))):
        for i in range(t.numel()):
            step = torch.zeros(t.numel(), dtype=torch.float64)
            step[i] = 1e-5
            step = step.view_as(t)
            slope = (at(t + step) - at(t - step)) / 2e-5
            # the third derivative times step^2 / 6, and float64's cancellation
            assert abs(slope - float(d.reshape(-1)[i])) <= 1e-7 * (1 + abs(slope))


def test_gated_grad_parts():
    """Of what d is kept in: 0 and 1 are one; two take as much workspace again."""
    def size(**kw):
        return _lib.moe_ep_gated_grad_workspace_bytes(grad_args(num_rows=100, **kw))
    assert size() == size(d_parts=1) and size(d_parts=2) - size() >= 100 * 64 * 2
    for bad in (-1, 3):
        assert grad(d_parts=bad) == INVALID
        assert status(_lib.moe_ep_gated_grad_workspace_bytes, grad_args(d_parts=bad)) == INVALID
    assert grad(num_rows=100, d_parts=2, workspace_bytes=size()) == INVALID
    assert grad(num_rows=0, d_parts=2, dgate_up=None, workspace=None, dout=None, pre=None, dx=None) == OK


@pytest.mark.parametrize("parts", [0, 3, None])
def test_gated_refuses_other_parts(parts):
    with pytest.raises(ValueError, match="grad_parts"):
        gated_linear(bf16(2, 64), bf16(16, 64), grad_parts=parts)
