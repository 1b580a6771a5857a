"""gated_linear's gradients with dgate and dup as two numbers of x's type each,
against the float64 forms, and how far either choice is from them."""

from __future__ import annotations

import pytest
import torch

from combine_token_dest_amd import gated_linear
from tests import dense_ref as ref
from tests.test_gpu_dense_gated import SIZES, make
from tests.test_gpu_experts import close, rand

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def want_grads(x, w, dh, dtype):
    """(dx, its bound, dw, its bound) of float64 with d in two parts: as in
    dense_ref.gated_grad, but for d's rounding.  Rounding the rest of a half step
    leaves a half step of it, 2^-16 of d in bfloat16 and 2^-22 in float16; float16's
    rest is kept times 2^11 in steps of 2^-24, and d's largest is at least 2^14: 2^-50
    of it."""
    x, w, dh = x.double(), w.double(), dh.double()
    g, u, _, tg, tu, _ = ref.gated(x, w)
    s1, silu = ref.silu_slope(g), g * ref.sigmoid(g)
    d = torch.cat((dh * u * s1, dh * silu), 1)
    more = (10 + 2 * g.abs()) * ref.U
    td = torch.cat((dh.abs() * ((1.1 + more) * tu + 0.51 * (u.abs() + tu) * tg + more * u.abs() * (s1.abs() + 0.2)),
                    dh.abs() * (1.1 * tg + more * silu.abs()) + 1e-36), 1)
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -11
    td = td + half ** 2 * (d.abs() + td) + (d.abs().max() * 2.0 ** -50 if dtype == F16 else ref.HALF_TINY[dtype])
    dx, t1 = ref.matmul(d, w.t())
    dw, t2 = ref.matmul(d.t(), x.t())
    # twice the additions, of magnitudes that add up to at most (1 + 2 half) of one part's
    t1 = 2 * t1 * (1 + 2.0 ** -6) + td @ w.abs()
    t2 = 2 * t2 * (1 + 2.0 ** -6) + td.t() @ x.abs()
    return dx, ref.rounded(dx, t1, dtype), dw, ref.rounded(dw, t2, dtype)


def grads(x, w, dh, parts, out_dtype=None):
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    h = gated_linear(gx, gw, grad_parts=parts, out_dtype=out_dtype)
    return (h.detach(), *torch.autograd.grad(h, (gx, gw), dh.cuda()))


def check(got, x, w, dh, dtype):
    want = want_grads(x, w, dh, dtype)
    close(got[1], want[0], want[1], "dx")
    close(got[2], want[2], want[3], "dgate_up")


# one to three tiles of k and more in each of the products, aligned and not, whole and in parts of k
TILES = [(5506, 265, 65), (134, 264, 2744), (1081, 136, 3592), (516, 200, 3336), (35, 333, 2234), (35, 328, 2112),
         (132, 5682, 149), (134, 5456, 152), (5378, 1416, 40), (641, 5408, 72), (1058, 70, 16), (300, 3592, 1090),
         (170, 6648, 264), (129, 2048, 32), (192, 1024, 96), (257, 1024, 128), (4096, 2048, 1024), (2500, 1100, 1027)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,H,I", SIZES + TILES)
def test_two_parts(n, H, I, dtype):
    x, w, dh = make(n, H, I, dtype)
    got = grads(x, w, dh, 2)
    check(got, x, w, dh, dtype)
    assert got[1].dtype == dtype and got[2].dtype == dtype
    assert torch.equal(got[0], grads(x, w, dh, 1)[0])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_how_near_each_choice_is(dtype):
    """With two parts what is left is the results' own rounding; with one, d's
    comes beside it: two errors of a size, 1.4 times one."""
    x, w, dh = make(700, 520, 264, dtype)
    exact = want_grads(x, w, dh, dtype)[::2]
    near = [v.to(dtype).double() for v in exact]
    off = {p: [float((g.double().cpu() - v).norm() / (r - v).norm()) for g, v, r in zip(grads(x, w, dh, p)[1:], exact, near)]
           for p in (1, 2)}
    assert all(e <= 1.02 for e in off[2]), off
    assert all(1.2 <= e <= 1.7 for e in off[1]), off


def test_float32_results_and_one_gradient_alone():
    x, w, _ = make(50, 96, 72, F16)
    dh = rand(5, 50, 72, dtype=F32)
    check(grads(x, w, dh, 2, F32), x, w, dh, F16)
    want = want_grads(x, w, dh, F16)
    for i, t in enumerate((x, w)):
        a, b = x.cuda(), w.cuda()
        leaf = (a, b)[i].requires_grad_()
        g, = torch.autograd.grad(gated_linear(a, b, out_dtype=F32, grad_parts=2), leaf, dh.cuda())
        close(g, want[2 * i], want[2 * i + 1])


@pytest.mark.parametrize("xs,ws,scale", [(8.0, 8.0, 3e-7), (8.0, 8.0, 1e-3), (256.0, 2.0 ** -9, 1e4)])
def test_float16_gradients_outside_its_range(xs, ws, scale):
    """dgate and dup beyond 65504, or far below 2^-14, with dx inside (the last case's dgate_up is not)."""
    x, w = rand(1, 70, 128, dtype=F16, std=xs), rand(2, 128, 128, dtype=F16, std=ws)
    dh = rand(3, 70, 64, dtype=F32, std=scale)
    _, dx, dw = grads(x, w, dh, 2, F32)
    want = want_grads(x, w, dh, F16)
    for got, v, tol in ((dx, *want[:2]), (dw, *want[2:])):
        fits = v.abs() + tol < 65504
        assert got is dw or fits.double().mean() > 0.9
        assert ((got.double().cpu() - v).abs()[fits] <= tol[fits]).all()


@pytest.mark.parametrize("n", [3, 140])
def test_special_values(n):
    """An infinite gradient stays one (its rounding leaves nothing), in its own row."""
    x, w, dh = make(n, 72, 48, BF16)
    dh[1, 5] = float("inf")
    one, two = (grads(x, w, dh, p) for p in (1, 2))
    keep = [r for r in range(n) if r != 1]
    want = want_grads(x[keep], w, dh[keep], BF16)
    close(two[1][keep], want[0], want[1])
    for a, b in zip(one, two):
        assert torch.equal(a.isfinite(), b.isfinite()) and torch.equal(a.isnan(), b.isnan())


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=F16, device="cuda").requires_grad_(), rand(1, 32, 64, dtype=F16).cuda().requires_grad_()
    h = gated_linear(x, w, grad_parts=2)
    dx, dw = torch.autograd.grad(h, (x, w), torch.empty(0, 16, dtype=F16, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_strides_and_alignment():
    n, H, I = 200, 104, 48
    x, w, dh = make(n, H, I, BF16)
    xb, wb = torch.zeros(n, 2 * H + 8, dtype=BF16, device="cuda"), torch.zeros(2 * I, H + 9, dtype=BF16, device="cuda")
    xv, wv = xb[:, 1:1 + H], wb[:, 1:1 + H]
    xv.copy_(x), wv.copy_(w)
    xv, wv = xv.detach().requires_grad_(), wv.detach().requires_grad_()
    got = torch.autograd.grad(gated_linear(xv, wv, grad_parts=2), (xv, wv), dh.cuda())
    check((None, *got), x, w, dh, BF16)


@pytest.mark.parametrize("n", [4, 150])
def test_graph(n):
    H, I = 264, 136
    sets = [make(n, H, I, F16, seed=10 * i) for i in range(3)]
    gx, gw, gd = (t.cuda() for t in sets[0])
    gx.requires_grad_(), gw.requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.autograd.grad(gated_linear(gx, gw, grad_parts=2), (gx, gw), gd)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = gated_linear(gx, gw, grad_parts=2)
        dx, dw = torch.autograd.grad(h, (gx, gw), gd)
    for x, w, dh in sets:
        with torch.no_grad():
            gx.copy_(x), gw.copy_(w), gd.copy_(dh)
        graph.replay()
        torch.cuda.synchronize()
        check((h, dx, dw), x, w, dh, F16)
        gated_linear(gx.detach(), gw.detach())
        torch.cuda.synchronize()


def test_same_bits_each_time():
    x, w, dh = make(300, 520, 264, BF16)
    first = grads(x, w, dh, 2)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, grads(x, w, dh, 2)))
