"""gated_linear on the GPU, forward and backward, against its float64 forms
(tests/dense_ref.py): types, sizes from one row to the largest tiles, odd and
strided matrices, special values, streams and graphs."""

from __future__ import annotations

import math

import pytest
import torch

from combine_token_dest_amd import gated_linear
from tests import dense_ref as ref
from tests.test_gpu_experts import close, rand

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make(n, H, I, dtype, seed=1):
    return (rand(seed, n, H, dtype=dtype), rand(seed + 1, 2 * I, H, dtype=dtype, std=1.5 / math.sqrt(H)),
            rand(seed + 2, n, I, dtype=dtype))


def check_forward(got, x, w):
    _, _, h, _, _, th = ref.gated(x, w)
    close(got, h, ref.rounded(h, th, got.dtype), "h")


def check_grads(dx, dw, x, w, dh, dtype):
    want = ref.gated_grad(x, w, dh, dtype)
    close(dx, want[0], want[1], "dx")
    close(dw, want[2], want[3], "dgate_up")


SIZES = [(1, 8, 8), (1, 7168, 64), (2, 64, 1000), (3, 100, 37), (5, 1030, 9), (16, 256, 24), (17, 64, 64),
         (33, 129, 40), (64, 512, 128), (48, 1000, 72), (49, 264, 4200), (40, 72, 4104), (65, 200, 264), (127, 4100, 64), (129, 264, 136), (257, 520, 300),
         (300, 64, 8), (1000, 72, 200)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,H,I", SIZES)
def test_forward(n, H, I, dtype):
    x, w, _ = make(n, H, I, dtype)
    check_forward(gated_linear(x.cuda(), w.cuda()), x, w)
    check_forward(gated_linear(x.cuda(), w.cuda(), out_dtype=F32), x, w)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,H,I", SIZES)
def test_training(n, H, I, dtype):
    x, w, dh = make(n, H, I, dtype)
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    h = gated_linear(gx, gw)
    check_forward(h.detach(), x, w)
    dx, dw = torch.autograd.grad(h, (gx, gw), dh.cuda())
    assert dx.dtype == dtype and dw.dtype == dtype
    check_grads(dx, dw, x, w, dh, dtype)


@pytest.mark.parametrize("n,H,I", [(4096, 136, 2048), (4100, 4096, 32), (70, 4096, 2056), (513, 1160, 520)])
def test_largest_tiles(n, H, I):
    """Enough tiles of 256 x 256 for the whole chip, forward or backward."""
    x, w, dh = make(n, H, I, BF16)
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    h = gated_linear(gx, gw)
    check_forward(h.detach(), x, w)
    check_grads(*torch.autograd.grad(h, (gx, gw), dh.cuda()), x, w, dh, BF16)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,H,I", [
    (5506, 265, 65), (134, 264, 2744), (1081, 136, 3592), (516, 200, 3336), (35, 333, 2234), (35, 328, 2112),
    (132, 5682, 149), (134, 5456, 152), (5378, 1416, 40), (641, 5408, 72), (34, 68, 1301), (34, 64, 1304),
    (1058, 70, 16), (300, 139, 2732), (300, 3592, 1090), (170, 6648, 264)])
def test_every_kind_of_tile(n, H, I, dtype):
    """Each size of tiles, aligned and not, whole and in parts of k, in each
    of the three products."""
    x, w, dh = make(n, H, I, dtype)
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    h = gated_linear(gx, gw)
    check_forward(h.detach(), x, w)
    check_grads(*torch.autograd.grad(h, (gx, gw), dh.cuda()), x, w, dh, dtype)


@pytest.mark.parametrize("which", ["x", "gate_up"])
def test_one_gradient_alone(which):
    x, w, dh = make(40, 96, 56, BF16)
    gx, gw = x.cuda().requires_grad_(which == "x"), w.cuda().requires_grad_(which == "gate_up")
    g, = torch.autograd.grad(gated_linear(gx, gw), gx if which == "x" else gw, dh.cuda())
    want = ref.gated_grad(x, w, dh, BF16)
    close(g, *(want[:2] if which == "x" else want[2:]), which)


def test_float32_result_and_its_gradient():
    x, w, _ = make(50, 96, 72, F16)
    dh = rand(5, 50, 72, dtype=F32)
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    h = gated_linear(gx, gw, out_dtype=F32)
    assert h.dtype == F32
    check_grads(*torch.autograd.grad(h, (gx, gw), dh.cuda()), x, w, dh, F16)


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF16, device="cuda").requires_grad_()
    w = rand(1, 32, 64).cuda().requires_grad_()
    h = gated_linear(x, w)
    assert h.shape == (0, 16)
    dx, dw = torch.autograd.grad(h, (x, w), torch.empty(0, 16, dtype=BF16, device="cuda"))
    assert dx.shape == (0, 64) and dw.shape == (32, 64) and (dw == 0).all()
    # float16 has a factor that only rows set
    x16 = torch.empty(0, 64, dtype=F16, device="cuda").requires_grad_()
    w16 = rand(1, 32, 64, dtype=F16).cuda().requires_grad_()
    _, dw = torch.autograd.grad(gated_linear(x16, w16), (x16, w16), torch.empty(0, 16, dtype=F16, device="cuda"))
    assert (dw == 0).all()


@pytest.mark.parametrize("n", [6, 200])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_strides_and_alignment(n, shift):
    """Rows of larger matrices that start at any element, and results of the caller's."""
    H, I = 104, 48
    x, w, dh = make(n, H, I, BF16)
    xb = torch.full((n, 2 * H + 8), math.nan, dtype=BF16, device="cuda")
    wb = torch.full((2 * I, H + 8 + shift), math.nan, dtype=BF16, device="cuda")
    db = torch.full((n, I + 9), math.nan, dtype=BF16, device="cuda")
    xv, wv, dv = xb[:, shift:shift + H], wb[:, shift:shift + H], db[:, shift:shift + I]
    xv.copy_(x.cuda()), wv.copy_(w.cuda()), dv.copy_(dh.cuda())
    out = torch.full((n, I + 5), 9.0, dtype=BF16, device="cuda")
    assert gated_linear(xv, wv, out=out[:, shift:shift + I]).data_ptr() == out[:, shift:].data_ptr()
    check_forward(out[:, shift:shift + I], x, w)
    assert (out[:, :shift] == 9).all() and (out[:, shift + I:] == 9).all()
    xv, wv = xv.detach().requires_grad_(), wv.detach().requires_grad_()
    check_grads(*torch.autograd.grad(gated_linear(xv, wv), (xv, wv), dv), x, w, dh, BF16)


def test_rows_behind_the_last_stay():
    n, H, I = 130, 64, 72
    x, w, _ = make(n, H, I, BF16)
    out = torch.full((n + 40, I), 5.0, dtype=BF16, device="cuda")
    gated_linear(x.cuda(), w.cuda(), out=out[:n])
    check_forward(out[:n], x, w)
    assert (out[n:] == 5).all()


def test_expanded_inputs_and_gradients():
    """One row for all, and a sum's gradient, whose elements are one number."""
    x, w, _ = make(1, 64, 40, BF16)
    n = 37
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    h = gated_linear(gx.expand(n, 64), gw)
    check_forward(h.detach(), x.expand(n, 64), w)
    dx, dw = torch.autograd.grad(h.float().sum(), (gx, gw))
    one = torch.ones(n, 40, dtype=BF16)
    want = ref.gated_grad(x.expand(n, 64), w, one, BF16)
    # autograd adds the n equal rows' gradients, in float32 or bfloat16: one rounding an addition at most
    close(dx, want[0].sum(0, keepdim=True), want[1].sum(0, keepdim=True) + n * 2.0 ** -8 * want[0].abs().sum(0, keepdim=True))
    close(dw, want[2], want[3])
    d = torch.autograd.grad(gated_linear(gx.expand(n, 64), gw), gw, torch.ones(40, n, dtype=BF16, device="cuda").t())[0]
    close(d, want[2], want[3])


@pytest.mark.parametrize("n", [3, 140])
def test_special_values_stay_in_their_rows(n):
    """An infinity or NaN in x reaches its own row of h and dx, and all of dgate_up."""
    x, w, dh = make(n, 72, 48, BF16)
    x[1, 5] = math.nan
    bad = x.clone()
    h = gated_linear(bad.cuda(), w.cuda())
    assert h[1].isnan().all()
    keep = [r for r in range(n) if r != 1]
    check_forward(h[keep], x[keep], w)
    gx, gw = bad.cuda().requires_grad_(), w.cuda().requires_grad_()
    dx, dw = torch.autograd.grad(gated_linear(gx, gw), (gx, gw), dh.cuda())
    assert dx[1].isnan().all() and dw.isnan().all()
    want = ref.gated_grad(x[keep], w, dh[keep], BF16)
    close(dx[keep], want[0], want[1])


@pytest.mark.parametrize("xs,ws,scale", [(8.0, 8.0, 3e-7), (8.0, 8.0, 1e-3), (256.0, 2.0 ** -9, 1e4)])
def test_float16_gradients_outside_its_range(xs, ws, scale):
    """dgate and dup beyond 65504, or far below 2^-14, with results inside."""
    n, H, I = 70, 128, 64
    x, w = rand(1, n, H, dtype=F16, std=xs), rand(2, 2 * I, H, dtype=F16, std=ws)
    dh = rand(3, n, I, dtype=F32, std=scale)
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    dx, dw = torch.autograd.grad(gated_linear(gx, gw, out_dtype=F32), (gx, gw), dh.cuda())
    want = ref.gated_grad(x, w, dh, F16)
    # dgate_up's terms reach 10^8 in the last case: a sum whose bound crosses float16's end may round to infinity
    fits = want[0].abs() + want[1] < 65504
    assert fits.double().mean() > 0.99
    assert ((dx.double().cpu() - want[0]).abs()[fits] <= want[1][fits]).all()
    fits = want[2].abs() + want[3] < 65504
    assert ((dw.double().cpu() - want[2]).abs()[fits] <= want[3][fits]).all()


def test_a_float16_gate_and_up_beyond_float16():
    """What is kept for the backward pass does not end at 65504."""
    n, H, I = 20, 64, 16
    x, w = rand(1, n, H, dtype=F16, std=300.0), rand(2, 2 * I, H, dtype=F16, std=100.0)
    w[:I] *= -2.0 ** -12
    dh = rand(3, n, I, dtype=F16, std=2.0 ** -10)
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    dx, _ = torch.autograd.grad(gated_linear(gx, gw, out_dtype=F32), (gx, gw), dh.float().cuda())
    want = ref.gated_grad(x, w, dh, F16)
    fits = want[0].abs() + want[1] < 65504
    assert fits.any() and ((dx.double().cpu() - want[0]).abs()[fits] <= want[1][fits]).all()


def test_past_32_bits():
    """Weights whose rows start more than 2^31 elements in."""
    n, H, I, stride = 3, 64, 8, 1 << 28
    x, w, dh = make(n, H, I, BF16)
    buf = torch.empty(15 * stride + H, dtype=BF16, device="cuda")
    wv = buf.as_strided((2 * I, H), (stride, 1))
    wv.copy_(w.cuda())
    check_forward(gated_linear(x.cuda(), wv), x, w)
    gx = x.cuda().requires_grad_()
    dx, = torch.autograd.grad(gated_linear(gx, wv), gx, dh.cuda())
    want = ref.gated_grad(x, w, dh, BF16)
    close(dx, want[0], want[1])


@pytest.mark.parametrize("n", [4, 150])
def test_streams_and_graph(n):
    """A captured training step, replayed with other inputs."""
    H, I = 264, 136
    sets = [make(n, H, I, F16, seed=10 * i) for i in range(3)]
    gx, gw, gd = (t.cuda() for t in sets[0])
    gx.requires_grad_(), gw.requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = torch.autograd.grad(gated_linear(gx, gw), (gx, gw), gd)
    s.synchronize()
    check_grads(*first, *sets[0], F16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = gated_linear(gx, gw)
        dx, dw = torch.autograd.grad(h, (gx, gw), gd)
    for x, w, dh in sets:
        with torch.no_grad():
            gx.copy_(x), gw.copy_(w), gd.copy_(dh)
        graph.replay()
        torch.cuda.synchronize()
        check_forward(h.detach(), x, w)
        check_grads(dx, dw, x, w, dh, F16)
        gated_linear(gx.detach(), gw.detach())
        torch.cuda.synchronize()


def test_no_second_derivatives():
    x, w, dh = (t.cuda().requires_grad_() for t in make(8, 64, 16, BF16))
    dx, = torch.autograd.grad(gated_linear(x, w), x, dh, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.float().sum().backward()


def test_weights_changed_before_the_backward_pass_are_noticed():
    x, w, dh = (t.cuda() for t in make(8, 64, 16, BF16))
    w.requires_grad_()
    h = gated_linear(x, w)
    with torch.no_grad():
        w.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(h, w, dh)


def test_inference_mode_and_leaves_through_a_module():
    """A down projection by torch behind it, gradients into .grad."""
    x, w, _ = make(20, 64, 24, BF16)
    down = rand(9, 64, 24)
    gx, gw, gd = (t.cuda().requires_grad_() for t in (x, w, down))
    with torch.inference_mode():
        check_forward(gated_linear(gx, gw), x, w)
    (gated_linear(gx, gw).float() @ gd.float().t()).sum().backward()
    dh = down.double().sum(0, keepdim=True).expand(20, 24)
    want = ref.gated_grad(x, w, dh, BF16)
    # the gradient of h arrives as bfloat16 of a float32 sum: one rounding more of each term
    more = 2.0 ** -8
    _, _, _, tg, tu, _ = ref.gated(x, w)
    d = torch.cat((dh.abs(), dh.abs()), 1) * 2 * (ref.gated(x, w)[1].abs().repeat(1, 2) + ref.gated(x, w)[0].abs().repeat(1, 2))
    close(gx.grad, want[0], want[1] + more * d @ w.double().abs())
    close(gw.grad, want[2], want[3] + more * d.t() @ x.double().abs())


def test_two_streams_at_once():
    sets = [make(90, 264, 72, BF16, seed=30 * i) for i in range(2)]
    dev = [[t.cuda() for t in s] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for (x, w, dh), st in zip(dev, streams):
            with torch.cuda.stream(st):
                a, b = x.detach().requires_grad_(), w.detach().requires_grad_()
                h = gated_linear(a, b)
                got.append((h.detach(), *torch.autograd.grad(h, (a, b), dh)))
    torch.cuda.synchronize()
    for i, (h, dx, dw) in enumerate(got):
        check_forward(h, *sets[i % 2][:2])
        check_grads(dx, dw, *sets[i % 2], BF16)


def test_same_bits_each_time():
    x, w, dh = (t.cuda() for t in make(300, 520, 264, BF16))
    x.requires_grad_(), w.requires_grad_()
    runs = []
    for _ in range(3):
        h = gated_linear(x, w)
        runs.append((h.detach(), *torch.autograd.grad(h, (x, w), dh)))
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))
