"""rms_norm on the GPU against its float64 form (tests/dense_ref.py): types,
sizes from one row to many and from eight columns to more than a workgroup
holds, strides, rows in place, special values, streams and graphs, and rows
on their way through an 8-bit dispatch."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from combine_token_dest_amd import MoEEp, rms_norm
from tests import dense_ref as ref
from tests.test_gpu_experts import close, rand

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


def check(x, w, residual=None, *, eps=EPS, eight=False, g=0, **kw):
    """Runs one call on the GPU and compares all it returns."""
    r = rms_norm(x.cuda(), w.cuda(), None if residual is None else residual.cuda(), eps=eps,
                 out_dtype=E4M3 if eight else None, group_size=g, **kw)
    torch.cuda.synchronize()
    verify(r, x, w, residual, eps, eight, g)
    return r


def verify(r, x, w, residual, eps=EPS, eight=False, g=0):
    y, tol = ref.norm(x, w, residual, eps)
    if residual is None:
        assert r.residual is None
    else:
        assert torch.equal(r.residual.cpu(), (x.float() + residual.float()).to(x.dtype))
    if not eight:
        assert r.scales is None and r.rows.dtype == x.dtype
        close(r.rows, y, ref.rounded(y, tol, x.dtype), "rows")
        return
    assert r.rows.dtype == E4M3 and r.rows.shape == x.shape
    q, scales = r.rows.cpu().to(torch.float64), r.scales.double().cpu()
    for i, part in enumerate(ref.groups_of(x.shape[1], g)):
        top = y[:, part].abs().amax(1)
        # y's six half steps and the quotient's; a scale may end at float32's smallest value
        assert ((scales[:, i] - top / 448).abs() <= 8 * ref.U * top / 448 + 2.0 ** -150).all()
        s = scales[:, i:i + 1]
        v = y[:, part] / s.clamp_min(1e-300)
        # half a step, and three roundings on the way to the quotient beside y's own
        tol_q = ref.e4m3_half_step(v * (1 + 2.0 ** -20)) * s + 10 * ref.U * y[:, part].abs()
        assert ((q[:, part] * s - y[:, part]).abs() <= tol_q).all()


@pytest.mark.parametrize("eight,g", [(False, 0), (True, 0), (True, 32), (True, 64), (True, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,H", [(1, 8), (1, 7168), (3, 100), (5, 4001), (2, 1024), (600, 264), (513, 4104),
                                 (1, 16384), (2, 32771), (520, 8200)])
def test_sizes(n, H, dtype, eight, g):
    x, res = rand(n + H, n, H, dtype=dtype, std=2.0), rand(n + H + 1, n, H, dtype=dtype, std=3.0)
    w = rand(7, H, dtype=dtype) * 0.2 + 1
    check(x, w, res, eight=eight, g=g)
    check(x, w.float() * 1.001, None, eight=eight, g=g)


def test_no_rows():
    r = rms_norm(torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda"),
                 torch.empty(0, 64, dtype=BF16, device="cuda"), out_dtype=E4M3, group_size=32)
    assert r.rows.shape == (0, 64) and r.scales.shape == (0, 2) and r.residual.shape == (0, 64)


def test_strided_rows_and_outputs_of_the_callers():
    n, H = 7, 203
    base, rbase = rand(1, n, 2 * H + 3), rand(2, n, H + 5)
    x, res, w = base[:, 3:3 + H], rbase[:, 1:1 + H], rand(3, H)
    gb, gr = base.cuda(), rbase.cuda()
    out = torch.full((n, H + 9), 77.0, dtype=BF16, device="cuda")
    rout = torch.full((n, H + 2), 77.0, dtype=BF16, device="cuda")
    r = rms_norm(gb[:, 3:3 + H], w.cuda(), gr[:, 1:1 + H], out=out[:, 2:2 + H], residual_out=rout[:, :H])
    assert r.rows.data_ptr() == out[:, 2:].data_ptr()
    verify(r, x, w, res)
    assert (out[:, :2] == 77).all() and (out[:, 2 + H:] == 77).all() and (rout[:, H:] == 77).all()
    out8 = torch.zeros(n, H + 13, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.full((n, 9), 5.0, device="cuda")
    r = rms_norm(gb[:, 3:3 + H], w.cuda(), out_dtype=E4M3, group_size=32, out=out8[:, 3:3 + H], scales=scales[:, 1:8])
    verify(r, x, w, None, eight=True, g=32)
    assert (scales[:, 0] == 5).all() and (scales[:, 8] == 5).all()
    assert (out8.view(torch.uint8)[:, :3] == 0).all() and (out8.view(torch.uint8)[:, 3 + H:] == 0).all()


def test_a_repeated_row():
    x, res, w = rand(1, 1, 96), rand(2, 5, 96), rand(3, 96)
    r = rms_norm(x.cuda().expand(5, 96), w.cuda(), res.cuda())
    verify(r, x.expand(5, 96), w, res)


@pytest.mark.parametrize("n,H", [(3, 300), (600, 520), (2, 40000)])
@pytest.mark.parametrize("eight", [False, True])
def test_in_place(n, H, eight):
    """residual_out is the residual; out is x (16 bits)."""
    x, res, w = rand(1, n, H), rand(2, n, H), rand(3, H)
    gx, gr = x.cuda(), res.cuda()
    if eight:
        r = rms_norm(gx, w.cuda(), gr, out_dtype=E4M3, group_size=128, residual_out=gr)
        assert torch.equal(gx.cpu(), x)
    else:
        r = rms_norm(gx, w.cuda(), gr, out=gx, residual_out=gr)
        assert r.rows is gx
    assert r.residual is gr
    verify(r, x, w, res, eight=eight, g=128 if eight else 0)
    # the outputs may also change places
    if not eight:
        gx, gr = x.cuda(), res.cuda()
        verify(rms_norm(gx, w.cuda(), gr, out=gr, residual_out=gx), x, w, res)


@pytest.mark.parametrize("std", [1e-30, 1e-4, 1e25, 5e37])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_small_and_large_values(std, eps):
    """No square overflows, and what is small beside eps keeps its bits (in 8
    bits as far as e4m3 with float32 scales holds them)."""
    x, w = rand(1, 3, 136, dtype=F32, std=std).to(BF16), rand(2, 136, dtype=F32)
    check(x, w, eps=eps)
    check(x, w, eps=eps, eight=True, g=64)
    check(x, w, eps=eps, eight=True)


@pytest.mark.parametrize("group", [0, 32, 64])
@pytest.mark.parametrize("k", [1, 3, 5, 7])
def test_middles_round_to_even(k, group):
    """Rows of a largest value 448 k with values k t, t in the middle of two
    e4m3 values: the quotients are t whatever the norm is, and t k has at most
    8 bits, so the whole path but for its roundings is exact."""
    H = 192
    t = torch.tensor([17.0, 19, 21, 23, 25, 27, 29, 31])
    t = torch.cat([t * 2.0 ** e for e in (-8, -4, 0, 3)] + [-t, -t / 2])[torch.arange(H) % 48]
    t[::32] = 448.0
    x = (t * k * torch.tensor([[1.0], [2.0 ** -20], [2.0 ** 30], [0.125]])).to(BF16)
    r = rms_norm(x.cuda(), torch.ones(H, dtype=BF16, device="cuda"), out_dtype=E4M3, group_size=group, eps=1e-6)
    assert (r.rows.cpu().float() == t.to(E4M3).float()).all()


def test_scales_below_the_smallest_normal():
    """Groups whose weight is tiny: the scale is subnormal or 0."""
    x = rand(1, 4, 256)
    w = torch.ones(256)
    w[64:128], w[128:192], w[192:] = 1e-42, 1e-45, 0.0
    r = rms_norm(x.cuda(), w.cuda(), out_dtype=E4M3, group_size=64)
    s, q = r.scales.cpu(), r.rows.cpu().float()
    assert (s[:, 3] == 0).all() and (q[:, 192:] == 0).all()
    y, tol = ref.norm(x, w, None, EPS)
    for i in range(3):
        part = slice(64 * i, 64 * i + 64)
        # float32's smallest step beside the relative ones, times what e4m3 multiplies it with
        near = (q[:, part].double() * s[:, i:i + 1].double() - y[:, part]).abs() <= \
            2.0 ** -4 * y[:, part].abs() + 448 * 2.0 ** -149
        assert near.all()
        assert q[:, part].isfinite().all()


def test_zero_rows_and_special_values():
    H = 256
    x = rand(1, 6, H)
    x[0] = 0
    x[1, 5] = math.inf
    x[2, 200] = math.nan
    x[3, 7] = -math.inf
    w = torch.ones(H, dtype=BF16)
    r = rms_norm(x.cuda(), w.cuda()).rows.cpu()
    assert (r[0] == 0).all()
    for i, c in ((1, 5), (3, 7)):            # the mean is infinite: others are 0, the infinity has no value
        assert r[i, c].isnan() and (r[i, :c] == 0).all() and (r[i, c + 1:] == 0).all()
    assert r[2].isnan().all() and r[4:].isfinite().all()
    r = rms_norm(x.cuda(), w.cuda(), out_dtype=E4M3, group_size=64)
    s, q = r.scales.cpu(), r.rows.cpu().float()
    assert (s[0] == 0).all() and (q[0] == 0).all()
    assert s[1, 0].isnan() and q[1, :64].isnan().all() and (s[1, 1:] == 0).all() and (q[1, 64:] == 0).all()
    assert s[2].isnan().all() and q[2].isnan().all()
    verify(type(r)(r.rows[4:], r.scales[4:], None), x[4:], w, None, eight=True, g=64)


def test_past_32_bits():
    """Rows that start more than 2^31 elements in."""
    n, H, stride = 3, 512, (1 << 30) + 64
    w = rand(3, H)
    x = rand(1, n, H)
    buf = torch.empty((n - 1) * stride + H, dtype=BF16, device="cuda")
    rows = buf.as_strided((n, H), (stride, 1))
    rows.copy_(x.cuda())
    verify(rms_norm(rows, w.cuda(), out=rows), x, w, None)


def test_more_rows_than_a_launch():
    """2^25 rows are a launch's most at 64 threads each."""
    n, H = (1 << 25) + 1000, 8
    x = torch.empty(n, H, dtype=BF16, device="cuda").fill_(1.0)
    w = rand(3, H)
    at = torch.tensor([0, 1, 12345, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, n - 1])
    some = rand(4, len(at), H)
    x[at.cuda()] = some.cuda()
    r = rms_norm(x, w.cuda(), x, out_dtype=E4M3)
    picked = type(r)(r.rows.view(torch.uint8)[at.cuda()].view(E4M3), r.scales[at.cuda()], r.residual[at.cuda()])
    verify(picked, some, w, some, eight=True)


def test_streams_and_graph():
    n, H = 64, 7168
    xs = [rand(i, n, H) for i in range(3)]
    res, w = rand(9, n, H), rand(10, H)
    gx, gr, gw = xs[0].cuda(), res.cuda(), w.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = rms_norm(gx, gw, gr, out_dtype=E4M3, group_size=128)
    s.synchronize()
    verify(r, xs[0], w, res, eight=True, g=128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = rms_norm(gx, gw, gr, out_dtype=E4M3, group_size=128)
    for x in xs:
        gx.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        verify(r, x, w, res, eight=True, g=128)
        rms_norm(gx, gw)
        torch.cuda.synchronize()


def test_rows_through_an_eight_bit_dispatch():
    """The norm's rows and scales are dispatch's hidden rows and scale rows."""
    ep, E, k, n, H = 4, 16, 2, 9, 384
    moe = MoEEp(ep, E, k, n, H, hidden_row_bytes=H, scale_row_bytes=H // 128 * 4)
    w = rand(1, H)
    normed, ids, weights = [], [], []
    for s in range(ep):
        r = rms_norm(rand(s, n, H).cuda(), w.cuda(), rand(50 + s, n, H).cuda(), out_dtype=E4M3, group_size=128)
        normed.append(r)
        ids.append(torch.from_numpy(np.random.RandomState(s).randint(0, E, (n, k)).astype(np.int32)).cuda())
        weights.append(torch.ones(n, k, device="cuda"))
    got = moe.dispatch([r.rows for r in normed], ids, weights, hidden_states_scale=[r.scales for r in normed])
    torch.cuda.synchronize()
    for d in range(ep):
        for s in range(ep):
            for t in range(n):
                if (ids[s][t].cpu() // (E // ep) == d).any():
                    row = s * got[d].tokens_per_rank + t
                    assert torch.equal(got[d].hidden[row].view(torch.uint8), normed[s].rows[t].view(torch.uint8))
                    assert torch.equal(got[d].hidden_scale[row], normed[s].scales[t])
    moe.destroy()
