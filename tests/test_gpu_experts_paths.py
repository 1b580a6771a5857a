"""The expert-side operators' ways through their kernels, each at the sizes
that lead there: many experts and several passes of 2048 tokens in the kernels
for few tokens to an expert, a router's choice over several passes, and the
kernels for many tokens at real widths.  Against float64, with a bound that
covers the longest chain of additions that any of the kernels has."""

from __future__ import annotations

import pytest
import torch

import combine_token_dest_amd as pkg
from combine_token_dest_amd import Router, expert_linear, moe_layer, route
from tests import experts_ref as ref
from tests.test_gpu_experts import BF16, F16, F32, close, gen, make_weight, rand

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23


def chain(K, g, parts=1):
    """Additions one after another in a sum over K columns: 32 inside a matrix
    instruction; an instruction for every 32 columns and part in one wave (the
    kernels that share the sum between waves have fewer), two for 4-bit weights
    and for float16 ones in parts; one for every 4-bit group and its scale; the
    waves' 8 parts."""
    return 32 + 2 * parts * (K // 32 + 1) + (2 * (K // g + 1) if g else 0) + 8


def product(w, x, adds):
    """(x w^T, bound): each addition is off by at most a step of a partial sum,
    and none is larger than the sum of the terms' magnitudes."""
    W, mag = w
    return x @ W.t(), adds * STEP * (x.abs() @ mag.t())


def linear64(x, rw, ids, offset, g, out_dtype):
    n, N, K = x.shape[0], rw.shape[1], rw.shape[2]
    y, tol = torch.zeros(2, n, N, dtype=torch.float64)
    for e in range(rw.shape[0]):
        rows = (ids == e + offset).nonzero().flatten()
        if len(rows):
            y[rows], tol[rows] = product(rw.expert(e), x[rows].double(), chain(K, g))
    return y, ref.rounded(y, tol, out_dtype)


def layer64(x, rg, rd, ids, weights, offset, gg, gd, out_dtype):
    """The layer and its bound: silu's slope is below 1.1; exp, sum, quotient
    and product are 8 half steps; the activation between is whole; a token's
    experts are added to their weighted sum with a step each."""
    n, H, I = x.shape[0], x.shape[1], rd.shape[2]
    y, tol, size = torch.zeros(3, n, H, dtype=torch.float64)
    for e in range(rg.shape[0]):
        rows, slots = (ids == e + offset).nonzero(as_tuple=True)
        if not len(rows):
            continue
        gu, t = product(rg.expert(e), x[rows].double(), chain(H, gg))
        gate, up, dg, du = gu[:, :I], gu[:, I:], t[:, :I], t[:, I:]
        silu = gate / (1 + torch.exp(-gate))
        act = silu * up
        da = 1.1 * (up.abs() + du) * dg + silu.abs() * du + 8 * 2.0 ** -24 * act.abs()
        W, mag = rd.expert(e)
        v, dv = product((W, mag), act, chain(I, gd, 3))
        w = weights[rows, slots].double().unsqueeze(1)
        y.index_add_(0, rows, w * v)
        tol.index_add_(0, rows, w.abs() * (dv + da @ W.abs().t()))
        size.index_add_(0, rows, w.abs() * (act.abs() @ mag.t()))
    tol += (ids.shape[1] + 8) * STEP * size
    return y, ref.rounded(y, tol, out_dtype)


def is_wide(n, E, k, H, I, g):
    """Whether the library takes its kernels for many tokens: these need room
    for each pair's float32 output beside the plan and the activations."""
    n = min(n, 2048)
    pairs, slots = n * k, min(n * k, E)
    other = sum(-(-b // 256) * 256 for b in (slots * 16 * 4, slots * n * 8, 6 * pairs * -(-I // 16) * 16))
    size = pkg.moe_layer_workspace_bytes(n, k, E, H, I, group_size=g)
    assert size in (other, other + -(-pairs * -(-H // 16) * 64 // 256) * 256)
    return size > other


@pytest.mark.parametrize("g", [0, 32])
@pytest.mark.parametrize("n,E,k", [(300, 1024, 3), (1300, 1024, 1), (200, 700, 5)])
def test_narrow_layer_of_more_experts_than_threads(n, E, k, g):
    """More than 512 experts or pairs that may have tokens: the down product
    goes through its plan in several rounds."""
    H, I = 48, 24
    print(f"[paths] narrow n={n} E={E} k={k} g={g}", flush=True)
    assert not is_wide(n, E, k, H, I, g) and min(n * k, E) > 512
    x = rand(1, n, H)
    rg, gu = make_weight(3, E, 2 * I, H, BF16, g)
    rd, dn = make_weight(4, E, H, I, BF16, g)
    ids = torch.stack([torch.randperm(E, generator=gen(s))[:k] for s in range(n)]).int()
    w = torch.rand(n, k, generator=gen(6))
    want, tol = layer64(x, rg, rd, ids, w, 0, g, g, F32)
    close(moe_layer(x.cuda(), gu, dn, ids.cuda(), w.cuda(), out_dtype=F32), want, tol)


@pytest.mark.parametrize("n", [2050, 4096, 4100])
def test_narrow_kernels_over_several_passes(n):
    """Few tokens to an expert in each pass of 2048, the last pass short; in
    place, in strided rows."""
    E, k, H, I, offset = 1024, 1, 40, 24, 7
    print(f"[paths] narrow passes n={n}", flush=True)
    assert not is_wide(n, E, k, H, I, 0)
    wide_rows = rand(1, n, H + 8)
    x = wide_rows[:, 8:]
    rg, gu = make_weight(3, E, 2 * I, H, BF16, 0)
    rd, dn = make_weight(4, E, H, I, BF16, 0)
    ids = torch.randint(offset - 3, E + offset + 3, (n, k), generator=gen(2)).int()
    w = torch.rand(n, k, generator=gen(6))
    want, tol = layer64(x, rg, rd, ids, w, offset, 0, 0, BF16)
    dev = wide_rows.cuda()
    rows = dev[:, 8:]
    nbytes = pkg.moe_layer_workspace_bytes(n, k, E, H, I)
    ws = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    moe_layer(rows, gu, dn, ids.cuda(), w.cuda(), expert_offset=offset, out=rows, workspace=ws[:nbytes])
    close(rows, want, tol)
    assert torch.equal(dev[:, :8].cpu(), wide_rows[:, :8]) and (ws[nbytes:] == 0xFF).all()
    y, ytol = linear64(x, rg, ids[:, 0], offset, 0, F32)
    first = ids[:, 0].contiguous().cuda()
    close(expert_linear(wide_rows.cuda()[:, 8:], gu, first, expert_offset=offset, out_dtype=F32), y, ytol, "linear")


@pytest.mark.parametrize("E,g,many", [(1024, 0, False), (16, 0, True), (16, 64, True)])
@pytest.mark.parametrize("score,bias,groups", [("softmax", False, 1), ("sigmoid", True, 4)])
@pytest.mark.parametrize("n,k", [(2051, 1), (2056, 2), (2057, 1)])
def test_router_over_several_passes(E, g, many, score, bias, groups, n, k):
    """Logits of more than one pass: strided rows of them, a last pass of up to
    8 tokens that the first product's kernel routes itself where experts have
    few tokens (and of 9, which it does not); the same bits as route followed
    by the layer, and the definition."""
    H, I, R = 32, 24, 16 if many else 256
    print(f"[paths] router n={n} k={k} E={E} g={g} {score}", flush=True)
    assert is_wide(n, E, k, H, I, g) == many
    x = rand(1, n, H)
    rg, gu = make_weight(3, E, 2 * I, H, BF16, g)
    rd, dn = make_weight(4, E, H, I, BF16, g)
    logits = rand(5, n, R + 3, dtype=F32).cuda()[:, :R]
    r = Router(k, score, rand(3, R, dtype=F32, std=0.1).cuda() if bias else None, num_groups=groups,
               top_groups=max(1, groups // 2), scale=2.5, renormalize=k > 1)
    ids, w = route(logits, r)
    a = moe_layer(x.cuda(), gu, dn, ids, w)
    b = moe_layer(x.cuda(), gu, dn, router_logits=logits, router=r)
    assert torch.equal(a, b)
    want, tol = layer64(x, rg, rd, ids.cpu(), w.cpu(), 0, g, g, BF16)
    close(b, want, tol)


@pytest.mark.parametrize("g", [0, 64])
def test_wide_kernels_of_more_experts_than_threads(g):
    """Many tokens to each of more than 256 experts (which are not sorted by load)."""
    n, E, k, H, I = 2000, 300, 4, 72, 40
    print(f"[paths] wide E={E} g={g}", flush=True)
    assert is_wide(n, E, k, H, I, g)
    x = rand(1, n, H)
    rg, gu = make_weight(3, E, 2 * I, H, BF16, g)
    rd, dn = make_weight(4, E, H, I, BF16, g)
    ids = torch.stack([torch.randperm(E, generator=gen(s))[:k] for s in range(n)]).int()
    w = torch.rand(n, k, generator=gen(6))
    want, tol = layer64(x, rg, rd, ids, w, 0, g, g, F32)
    close(moe_layer(x.cuda(), gu, dn, ids.cuda(), w.cuda(), out_dtype=F32), want, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("g", [0, 32, 128])
@pytest.mark.parametrize("n,E,k,H,I", [(150, 4, 2, 4096, 1024), (90, 3, 1, 1000, 2056)])
def test_wide_kernels_at_real_widths(dtype, g, n, E, k, H, I):
    print(f"[paths] wide {dtype} g={g} n={n} H={H} I={I}", flush=True)
    assert is_wide(n, E, k, H, I, g)
    x = rand(1, n, H, dtype=dtype)
    rg, gu = make_weight(3, E, 2 * I, H, dtype, g)
    rd, dn = make_weight(4, E, H, I, dtype, g)
    ids = torch.stack([torch.randperm(E, generator=gen(s))[:k] for s in range(n)]).int()
    w = torch.rand(n, k, generator=gen(6))
    want, tol = layer64(x, rg, rd, ids, w, 0, g, g, F32)
    close(moe_layer(x.cuda(), gu, dn, ids.cuda(), w.cuda(), out_dtype=F32), want, tol)
    y, ytol = linear64(x, rg, ids[:, 0], 0, g, F32)
    close(expert_linear(x.cuda(), gu, ids[:, 0].contiguous().cuda(), out_dtype=F32), y, ytol, "linear")
