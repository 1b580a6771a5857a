"""route, expert_linear and moe_layer on the GPU against their float64 forms
(tests/experts_ref.py): types, sizes from one to odd and large, strides,
masks and invalid ids, special values, streams, graphs, and a decode step
through route, dispatch, the experts and combine."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import combine_token_dest_amd as pkg
from combine_token_dest_amd import MoEEp, Router, W4Weights, expert_linear, moe_layer, route
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(seed, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=gen(seed)) * std).to(dtype)


def make_weight(seed, E, N, K, dtype, g):
    """(reference form, what the operators take)."""
    std = 1.0 / math.sqrt(K)
    if g == 0:
        w = rand(seed, E, N, K, dtype=dtype, std=std)
        return ref.Dense(w), w.cuda()
    groups = -(-K // g)
    q = torch.randint(0, 16, (E, N, K), generator=gen(seed), dtype=torch.uint8)
    s = ((torch.rand(E, N, groups, generator=gen(seed + 1)) + 0.5) * std / 4.6).to(dtype)
    s[:, ::3] *= -1
    # spelled out for the layout: pack() may choose a smaller group for few columns
    return ref.W4(q, s, g), W4Weights._pack_groups(q.cuda(), s.cuda(), g)


def close(got, want, tol, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i} got {got[i]}, want {want[i]} "
                             f"+- {tol[i]}")


# -- route --------------------------------------------------------------------

def check_route(logits, router, bias=None, weights_rel=28 * 2.0 ** -24):
    """Ids equal; weights within 28 float32 half steps (a softmax sum of up
    to 1024 float32 exponentials: 2 for each, 1 for its argument, 16 + 6 + 2
    for the sum and the quotient; less in the other forms)."""
    kw = dict(score=router.score, num_groups=router.num_groups, top_groups=router.top_groups,
              group_top=router.group_top, renormalize=router.renormalize, scale=router.scale,
              invalid=router.invalid_expert_id)
    if bias is not None:
        router.bias = bias.cuda()
    ids, w = route(logits.cuda(), router)
    want_ids, want_w = ref.route(logits, router.top_k, bias=bias, **kw)
    n = logits.shape[0]
    want_ids = torch.tensor(want_ids, dtype=torch.int32).reshape(n, router.top_k)
    want_w = torch.tensor(want_w, dtype=torch.float64).reshape(n, router.top_k)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert torch.equal(ids.cpu(), want_ids)
    close(w, want_w, want_w.abs() * weights_rel + 2.0 ** -149, "weights")


@pytest.mark.parametrize("E,k", [(1, 1), (3, 3), (8, 2), (60, 4), (64, 8), (65, 6), (128, 8), (256, 8), (256, 17),
                                 (300, 64), (1024, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_route_sizes(E, k, score, dtype):
    print(f"[route] E={E} k={k} {score} {dtype}", flush=True)
    for n, renorm, scale in ((1, True, 1.0), (37, False, 2.5), (260, True, 2.5)):
        check_route(rand(E + n, n, E, dtype=dtype), Router(k, score, renormalize=renorm, scale=scale))


@pytest.mark.parametrize("E,G,top,per", [(256, 8, 4, 2), (64, 8, 3, 1), (60, 4, 2, 2), (8, 8, 4, 2), (512, 2, 1, 2),
                                         (1024, 64, 16, 2)])
@pytest.mark.parametrize("score,with_bias", [("softmax", False), ("sigmoid", True), ("softmax", True)])
def test_route_groups_and_bias(E, G, top, per, score, with_bias):
    print(f"[route] groups E={E} G={G} {score} bias={with_bias}", flush=True)
    bias = rand(5, E, dtype=F32, std=0.05) if with_bias else None
    k = min(4, top * (E // G))
    for n in (1, 33):
        check_route(rand(E + n, n, E, dtype=F32),
                    Router(k, score, num_groups=G, top_groups=top, group_top=per, scale=2.5), bias)


@pytest.mark.parametrize("n", [2048, 5000])
def test_route_many_tokens(n):
    check_route(rand(n, n, 128, dtype=BF16), Router(8, renormalize=False))
    check_route(rand(n, n, 96, dtype=F32), Router(6, "sigmoid"))


def test_route_more_tokens_than_a_launch_has():
    n = 2 ** 26 + 5                       # at 64 lanes each, 2^32 threads and more
    pattern = rand(7, 64, 2, dtype=F16).cuda()
    logits = pattern[torch.arange(n, device="cuda") % 64]
    for r in (Router(1), Router(1, bias=torch.zeros(2, device="cuda"))):
        ids, w = route(logits, r)
        want_ids, want_w = route(pattern, r)
        at = torch.arange(n, device="cuda") % 64
        assert torch.equal(ids, want_ids[at]) and torch.equal(w, want_w[at])


def test_route_ties_go_to_the_lowest_index():
    logits = torch.randint(-1, 2, (64, 96), generator=gen(3)).to(BF16)
    check_route(logits, Router(12))
    check_route(logits, Router(12, "sigmoid"), torch.zeros(96))
    check_route(logits.float(), Router(12, "sigmoid", num_groups=8, top_groups=4))
    check_route(torch.zeros(3, 256), Router(8, num_groups=8, top_groups=2))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_closed_experts(score, groups):
    """-inf, NaN, +inf, the type's lowest value, and rows with too few open experts."""
    inf, nan = math.inf, math.nan
    low = torch.finfo(F32).min
    E = 16
    x = rand(9, 12, E, dtype=F32)
    x[0] = -inf
    x[1] = nan
    x[2, 1:] = -inf
    x[3, :] = low
    x[4, 5] = inf
    x[5, [3, 9]] = inf
    x[6, ::2] = nan
    x[7, :14] = -inf
    x[8] = low
    x[8, 7] = 1.0
    x[9] = inf
    x[10] = -200.0            # sigmoids far below float32's normal numbers
    for renorm in (True, False):
        r = dict(renormalize=renorm, num_groups=groups, top_groups=max(1, groups // 2), invalid_expert_id=99)
        check_route(x, Router(4, score, **r))
        bias = rand(2, E, dtype=F32, std=0.1)
        bias[[1, 6]] = -inf
        bias[11] = nan
        check_route(x, Router(4, score, **r), bias)


def test_route_strided_rows_and_given_outputs():
    wide = rand(4, 40, 200, dtype=F32)
    x = wide.cuda()[:, 7:135]
    ids = torch.full((40, 6), -7, dtype=torch.int32, device="cuda")
    w = torch.full((40, 6), -7.0, device="cuda")
    a, b = route(x, Router(6), topk_ids=ids, topk_weights=w)
    assert a is ids and b is w
    want, ww = ref.route(wide[:, 7:135], 6)
    assert ids.tolist() == want
    close(w, torch.tensor(ww, dtype=torch.float64), torch.tensor(ww, dtype=torch.float64) * 2.0 ** -20)
    one = route(x[:1].expand(5, -1), Router(6))[0]       # a repeated row
    assert one.tolist() == [want[0]] * 5
    empty = route(x[:0], Router(6))
    assert tuple(empty[0].shape) == (0, 6) and tuple(empty[1].shape) == (0, 6)


# -- expert_linear ------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("g", [0, 32, 64, 128])
@pytest.mark.parametrize("n,E,N,K", [(1, 1, 16, 128), (1, 4, 100, 64), (3, 2, 17, 72), (16, 5, 33, 513),
                                     (17, 3, 48, 200), (40, 2, 64, 1000), (70, 1, 40, 256), (130, 3, 20, 33),
                                     (5, 7, 1, 9), (6, 2, 5, 8), (2, 2, 31, 2049)])
def test_linear(dtype, g, n, E, N, K):
    print(f"[linear] {dtype} g={g} n={n} E={E} N={N} K={K}", flush=True)
    x = rand(n, n, K, dtype=dtype)
    rw, w = make_weight(K, E, N, K, dtype, g)
    offset = 3
    ids = torch.randint(offset - 1, offset + E + 1, (n,), generator=gen(n + E), dtype=torch.int32)
    for out_dtype in (dtype, F32):
        want, tol = ref.linear(x, rw, ids, offset, out_dtype)
        got = expert_linear(x.cuda(), w, ids.cuda(), expert_offset=offset, out_dtype=out_dtype)
        close(got, want, tol, f"ids {out_dtype}")
    want, tol = ref.linear(x, rw, None, 0, dtype)
    close(expert_linear(x.cuda(), w), want, tol, "one expert")


@pytest.mark.parametrize("g", [0, 64])
def test_linear_many_rows(g):
    """More rows than one pass takes, all of few experts."""
    n, E, N, K = 2200, 2, 24, 96
    x = rand(1, n, K)
    rw, w = make_weight(2, E, N, K, BF16, g)
    ids = torch.randint(0, E, (n,), generator=gen(3), dtype=torch.int32)
    want, tol = ref.linear(x, rw, ids, 0, BF16)
    close(expert_linear(x.cuda(), w, ids.cuda()), want, tol)
    want, tol = ref.linear(x, rw, None, 0, BF16)
    close(expert_linear(x.cuda(), w), want, tol)


@pytest.mark.parametrize("g", [0, 128])
def test_linear_strides_and_neighbours(g):
    """Strided, odd-aligned and repeated rows; what lies beside the output stays."""
    n, N, K = 9, 50, 131
    rw, w = make_weight(7, 2, N, K, F16, g)
    big = rand(8, n, K + 9, dtype=F16)
    x = big.cuda()[:, 3:3 + K]
    ids = torch.tensor([0, 1, 5, 0, 1, -1, 1, 1, 0], dtype=torch.int32)
    buf = torch.full((n + 2, N + 6), 77.0, dtype=F32, device="cuda")
    out = buf[1:n + 1, 5:5 + N]
    want, tol = ref.linear(big[:, 3:3 + K], rw, ids, 0, F32)
    assert expert_linear(x, w, ids.cuda(), out=out) is out
    close(out, want, tol)
    assert (buf[0] == 77).all() and (buf[-1] == 77).all() and (buf[:, :5] == 77).all() and (buf[:, 5 + N:] == 77).all()
    rep = expert_linear(x[:1].expand(4, -1), w)
    want, tol = ref.linear(big[:1, 3:3 + K].expand(4, -1), rw, None, 0, F16)
    close(rep, want, tol)


def test_linear_special_values_stay_in_their_rows():
    """NaN and infinity in one row, one expert's matrix, or padding touch no other result."""
    n, E, N, K = 20, 3, 40, 100
    rw, w = make_weight(1, E, N, K, BF16, 0)
    x = rand(2, n, K)
    ids = torch.arange(n, dtype=torch.int32) % E
    clean = expert_linear(x.cuda(), w, ids.cuda())
    x2, w2 = x.clone(), w.clone()
    x2[4] = math.nan
    x2[7, 3] = math.inf
    w2[1, 0, 0] = math.nan
    got = expert_linear(x2.cuda(), w2, ids.cuda())
    ok = [r for r in range(n) if r not in (4, 7)]
    same = torch.tensor([r for r in ok if ids[r] != 1])
    assert torch.equal(got[same], clean[same])
    rows1 = torch.tensor([r for r in ok if ids[r] == 1])
    assert torch.equal(got[rows1][:, 1:], clean[rows1][:, 1:]) and got[rows1][:, 0].isnan().all()
    assert got[4].isnan().all()
    want = (x2[7].double() @ w2[1].double().cpu().t()).to(F32)
    assert torch.equal(got[7].float().cpu().isnan(), want.isnan())
    assert torch.equal(got[7].float().cpu().isinf(), want.isinf())
    # 4 bits: padding scales of any value
    rw4, w4 = make_weight(3, 1, 20, 40, BF16, 32)
    want, tol = ref.linear(x[:5, :40], rw4, None, 0, F32)
    sc = w4.scales.clone()
    sc[:, :, 2:] = math.nan
    sc[:, 1, :, 4:] = math.inf
    data = w4.data.clone()
    close(expert_linear(x[:5, :40].cuda(), W4Weights(data, sc, 20, 40), out_dtype=F32), want, tol)


# -- moe_layer ----------------------------------------------------------------

def make_ids(seed, n, E, k, offset=0, extra=0):
    """Distinct ids per token, out of E + extra experts around the offset."""
    rng = np.random.default_rng(seed)
    lo = offset - extra // 2
    return torch.tensor(np.stack([rng.permutation(E + extra)[:k] for _ in range(n)]) if n else np.zeros((0, k)),
                        dtype=torch.int32) + lo


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("g", [0, 32, 64, 128])
@pytest.mark.parametrize("n,E,k,H,I", [(1, 8, 2, 64, 32), (1, 16, 8, 129, 40), (2, 4, 4, 200, 100), (7, 3, 2, 56, 17),
                                       (17, 8, 2, 128, 64), (33, 4, 3, 48, 130), (70, 2, 1, 40, 48),
                                       (131, 5, 2, 24, 20), (3, 2, 2, 9, 8), (2, 3, 2, 8, 11)])
def test_layer(dtype, g, n, E, k, H, I):
    print(f"[layer] {dtype} g={g} n={n} E={E} k={k} H={H} I={I}", flush=True)
    x = rand(n, n, H, dtype=dtype)
    rg, gu = make_weight(1, E, 2 * I, H, dtype, g)
    rd, dn = make_weight(2, E, H, I, dtype, g)
    ids = make_ids(n, n, E, k)
    w = torch.rand(n, k, generator=gen(4))
    for out_dtype in (dtype, F32):
        want, tol = ref.layer(x, rg, rd, ids, w, 0, dtype, out_dtype)
        close(moe_layer(x.cuda(), gu, dn, ids.cuda(), w.cuda(), out_dtype=out_dtype), want, tol, str(out_dtype))


@pytest.mark.parametrize("g", [0, 64])
def test_layer_of_one_rank(g):
    """Experts of other ranks, invalid rows, signed weights, no weights, ids named twice."""
    n, E, k, H, I, offset = 45, 6, 4, 72, 36, 12
    x = rand(1, n, H)
    rg, gu = make_weight(3, E, 2 * I, H, BF16, g)
    rd, dn = make_weight(4, E, H, I, BF16, g)
    ids = make_ids(5, n, E, k, offset, extra=12)
    ids[3] = -1
    ids[4] = 2 ** 31 - 1
    ids[5] = -2 ** 31
    ids[6] = offset + 2
    ids[7] = torch.tensor([offset, offset + 1, offset, offset], dtype=torch.int32)
    x[3] = math.nan                       # never read
    w = torch.randn(n, k, generator=gen(6))
    xr = x.clone()
    xr[3] = 0
    for weights in (w, None):
        want, tol = ref.layer(xr, rg, rd, ids, weights, offset, BF16, BF16)
        got = moe_layer(x.cuda(), gu, dn, ids.cuda(), None if weights is None else weights.cuda(),
                        expert_offset=offset)
        close(got, want, tol)
        assert (got[3:6] == 0).all()
    got64 = moe_layer(x.cuda(), gu, dn, ids.long().cuda().clamp(-1, 2 ** 30), w.cuda(), expert_offset=offset)
    assert torch.equal(got64, moe_layer(x.cuda(), gu, dn, ids.cuda().clamp(-1, 2 ** 30), w.cuda(), expert_offset=offset))


@pytest.mark.parametrize("n,E,k", [(2100, 4, 2), (300, 300, 3), (1000, 20, 9)])
def test_layer_many_tokens(n, E, k):
    """More tokens than a pass, and more experts than a block has threads' worth of slots."""
    H, I = 40, 24
    x = rand(1, n, H)
    rg, gu = make_weight(3, E, 2 * I, H, BF16, 0)
    rd, dn = make_weight(4, E, H, I, BF16, 32)
    ids = make_ids(2, n, E, k)
    w = torch.rand(n, k, generator=gen(6))
    want, tol = ref.layer(x, rg, rd, ids, w, 0, BF16, BF16)
    close(moe_layer(x.cuda(), gu, dn, ids.cuda(), w.cuda()), want, tol)


@pytest.mark.parametrize("g", [0, 64])
@pytest.mark.parametrize("H,I", [(64, 1100), (2200, 24)])
def test_layer_experts_of_unequal_load(H, I, g):
    """More workgroups than the card holds at once: experts of no, one and
    many tokens, equals among them, experts of other ranks, repeated ids."""
    n, k, E, offset = 500, 3, 32, 5
    x = rand(1, n, H)
    rg, gu = make_weight(3, E, 2 * I, H, BF16, g)
    rd, dn = make_weight(4, E, H, I, BF16, g)
    ids = torch.randint(0, 16, (n, k), generator=gen(2)) * torch.randint(0, 3, (n, k), generator=gen(3)) + offset - 2
    ids[:, 2] = torch.where(torch.arange(n) % 3 == 0, ids[:, 0], torch.full((n,), E + offset))
    ids = ids.int()
    w = rand(4, n, k, dtype=F32).abs()
    want, tol = ref.layer(x, rg, rd, ids, w, offset, BF16, BF16)
    close(moe_layer(x.cuda(), gu, dn, ids.cuda(), w.cuda(), expert_offset=offset), want, tol)
    y, ytol = ref.linear(x, rg, ids[:, 0], offset, BF16)
    close(expert_linear(x.cuda(), gu, ids[:, 0].cuda().contiguous(), expert_offset=offset), y, ytol, "linear")


@pytest.mark.parametrize("g", [0, 32])
@pytest.mark.parametrize("n,k", [(3, 4), (20, 8), (600, 4)])
def test_layer_ids_named_by_every_slot(n, k, g):
    """One expert in all slots of all tokens: more pairs than tokens, each token once."""
    E, H, I = 3, 40, 24
    x = rand(1, n, H)
    rg, gu = make_weight(3, E, 2 * I, H, BF16, g)
    rd, dn = make_weight(4, E, H, I, BF16, g)
    ids = torch.full((n, k), 1, dtype=torch.int32)
    w = torch.rand(n, k, generator=gen(6))
    want, tol = ref.layer(x, rg, rd, ids[:, :1], w.double().sum(1, keepdim=True), 0, BF16, BF16)
    # the k weights are added in float32 first
    tol = tol + k * 2.0 ** -24 * want.abs()
    close(moe_layer(x.cuda(), gu, dn, ids.cuda(), w.cuda()), want, tol)
    assert torch.equal(moe_layer(x.cuda(), gu, dn, ids.cuda() + 7, w.cuda()), torch.zeros(n, H, dtype=BF16, device="cuda"))


@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("score,bias,groups", [("softmax", False, 1), ("sigmoid", True, 4)])
def test_layer_routed_inside(n, score, bias, groups):
    """Logits in, the same bits as route followed by the layer."""
    E, k, H, I = 32, 4, 64, 48
    x = rand(1, n, H, dtype=F16).cuda()
    _, gu = make_weight(3, E, 2 * I, H, F16, 0)
    _, dn = make_weight(4, E, H, I, F16, 128)
    logits = rand(n, n, E, dtype=F32)
    logits[0, 3:] = -math.inf             # fewer open experts than slots
    logits = logits.cuda()
    r = Router(k, score, rand(3, E, dtype=F32, std=0.1).cuda() if bias else None, num_groups=groups,
               top_groups=max(1, groups // 2), scale=2.5)
    ids, w = route(logits, r)
    a = moe_layer(x, gu, dn, ids, w)
    b = moe_layer(x, gu, dn, router_logits=logits, router=r)
    assert torch.equal(a, b) and not a.isnan().any()


@pytest.mark.parametrize("n,E,k", [(8, 256, 8), (9, 256, 7), (8, 40, 9), (1, 256, 64), (3, 257, 5), (2, 3, 3)])
@pytest.mark.parametrize("dtype,g", [(BF16, 0), (F16, 32)])
def test_layer_routes_a_few_tokens_itself(n, E, k, dtype, g):
    """Up to 8 tokens, 64 pairs and 256 experts, and one past each; the experts
    of one rank, logits of each type in strided rows, NaN and ties among them."""
    H, I, here, offset = 72, 40, max(1, E // 4), E // 2
    x = rand(1, n, H, dtype=dtype).cuda()
    _, gu = make_weight(3, here, 2 * I, H, dtype, g)
    _, dn = make_weight(4, here, H, I, dtype, g)
    for i, (score, bias, groups, t) in enumerate([("softmax", False, 1, F32), ("softmax", False, 1, BF16),
                                                  ("sigmoid", True, 4, F16), ("softmax", True, 2, F32)]):
        if E % groups or k > E // groups:
            groups = 1
        logits = rand(E + i, n, E + 3, dtype=t)
        logits[-1, ::2] = logits[-1, 0]
        logits[0, E - 1] = math.nan
        logits[0, 0] = -math.inf
        logits = logits.cuda()[:, :E]
        r = Router(k, score, rand(3, E, dtype=F32, std=0.1).cuda() if bias else None, num_groups=groups,
                   top_groups=max(1, groups // 2), renormalize=i % 2 == 0, scale=2.5)
        ids, w = route(logits, r)
        a = moe_layer(x, gu, dn, ids, w, expert_offset=offset)
        b = moe_layer(x, gu, dn, router_logits=logits, router=r, expert_offset=offset)
        assert torch.equal(a, b) and not b.isnan().any(), (score, t)


def test_layer_in_place_strides_and_workspace():
    n, E, k, H, I = 5, 4, 2, 50, 30
    rg, gu = make_weight(3, E, 2 * I, H, BF16, 0)
    rd, dn = make_weight(4, E, H, I, BF16, 0)
    big = rand(1, n, H + 7)
    ids, w = make_ids(2, n, E, k), torch.rand(n, k, generator=gen(6))
    want, tol = ref.layer(big[:, 3:3 + H], rg, rd, ids, w, 0, BF16, BF16)
    dev = big.cuda()
    x = dev[:, 3:3 + H]
    nbytes = pkg.moe_layer_workspace_bytes(n, k, E, H, I)
    ws = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN bits in every type
    got = moe_layer(x, gu, dn, ids.cuda(), w.cuda(), workspace=ws[:nbytes])
    close(got, want, tol)
    assert (ws[nbytes:] == 0xFF).all()
    close(moe_layer(x, gu, dn, ids.cuda(), w.cuda(), out=x), want, tol, "in place")
    assert torch.equal(dev[:, :3].cpu(), big[:, :3]) and torch.equal(dev[:, 3 + H:].cpu(), big[:, 3 + H:])


def test_no_tokens():
    """Zero rows: nothing is launched, the results are empty."""
    w = rand(2, 2, 32, 64).cuda()
    dn = rand(4, 2, 64, 16).cuda()
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert tuple(expert_linear(x, w).shape) == (0, 32)
    assert tuple(expert_linear(x, w, ids[:, 0].contiguous()).shape) == (0, 32)
    assert tuple(moe_layer(x, w, dn, ids).shape) == (0, 64)
    assert tuple(moe_layer(x, w, dn, router_logits=torch.empty(0, 2, device="cuda"), router=Router(1)).shape) == (0, 64)


@pytest.mark.parametrize("g", [0, 32])
def test_offsets_past_32_bits(g):
    """The last of experts whose weights, and rows whose inputs and outputs, lie beyond 4 GiB."""
    E, N, K = (40, 8192, 8192) if g == 0 else (130, 8192, 8192)
    dense = rand(1, 1, N, K)[0]
    if g == 0:
        w = torch.empty(E, N, K, dtype=BF16, device="cuda")
        w[E - 1] = dense.cuda()
        rw = ref.Dense(dense.unsqueeze(0))
        assert w.numel() * 2 > 2 ** 32
    else:
        rw, one = make_weight(5, 1, N, K, BF16, g)
        data = torch.empty(E, *one.data.shape[1:], dtype=torch.uint8, device="cuda")
        sc = torch.empty(E, *one.scales.shape[1:], dtype=BF16, device="cuda")
        data[E - 1], sc[E - 1] = one.data[0], one.scales[0]
        w = W4Weights(data, sc, N, K)
        assert data.numel() > 2 ** 32
    far = torch.zeros(3, 2 ** 30, dtype=BF16, device="cuda")          # rows 2 GiB apart
    x = far[:, 5:5 + K]
    host = rand(2, 3, K)
    x.copy_(host)
    out = far[:, 2 ** 20:2 ** 20 + N]
    ids = torch.full((3,), E - 1, dtype=torch.int32, device="cuda")
    want, tol = ref.linear(host, rw, torch.zeros(3, dtype=torch.int32), 0, BF16)
    # (x and out interleave, which the overlap check refuses)
    with pytest.raises(pkg.MoeEpError, match="overlap"):
        expert_linear(x, w, ids, out=out)
    close(expert_linear(x, w, ids), want, tol, "x")
    close(expert_linear(host.cuda(), w, ids, out=out), want, tol, "out")


def test_layer_large_float16_activations():
    """Activations past float16's largest value are kept by the two parts."""
    n, H, I = 2, 16, 16
    x = torch.full((n, H), 8.0, dtype=F16)
    gu = torch.full((1, 2 * I, H), 2.0, dtype=F16)            # gate = up = 256: act = 65536
    dn = torch.full((1, H, I), 2.0 ** -10, dtype=F16)
    out = moe_layer(x.cuda(), gu.cuda(), dn.cuda(), torch.zeros(n, 1, dtype=torch.int32, device="cuda"))
    assert (out == 65536 * 16 * 2.0 ** -10).all()


def test_layer_special_values_stay_in_their_tokens():
    n, E, k, H, I = 20, 4, 2, 48, 32
    _, gu = make_weight(3, E, 2 * I, H, BF16, 0)
    _, dn = make_weight(4, E, H, I, BF16, 0)
    x = rand(1, n, H)
    ids = torch.stack([torch.arange(n) % E, (torch.arange(n) + 1) % E], 1).to(torch.int32)
    w = torch.rand(n, k, generator=gen(6)).cuda()
    clean = moe_layer(x.cuda(), gu, dn, ids.cuda(), w)
    x[5] = math.inf
    gu2, dn2 = gu.clone(), dn.clone()
    gu2[2, 0, 0] = math.nan
    dn2[2, :, 1] = math.inf
    got = moe_layer(x.cuda(), gu2, dn2, ids.cuda(), w)
    free = torch.tensor([t for t in range(n) if t != 5 and 2 not in ids[t].tolist()])
    assert torch.equal(got[free], clean[free])
    hit = torch.tensor([t for t in range(n) if 2 in ids[t].tolist()])
    assert got[hit].isnan().all()


def test_same_bits_again_and_on_another_stream():
    """Twice the same bits; two streams at once with their own workspaces."""
    n, E, k, H, I = 24, 16, 4, 256, 128
    _, gu = make_weight(3, E, 2 * I, H, BF16, 64)
    _, dn = make_weight(4, E, H, I, BF16, 64)
    xs = [rand(s, n, H).cuda() for s in range(2)]
    ls = [rand(s + 9, n, E, dtype=F32).cuda() for s in range(2)]
    r = Router(k)
    want = [moe_layer(x, gu, dn, router_logits=l, router=r) for x, l in zip(xs, ls)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(moe_layer(xs[i], gu, dn, router_logits=ls[i], router=r))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_graph_replays():
    """route, expert_linear and moe_layer captured together and replayed on
    new inputs, with eager calls of the same operators between the replays."""
    n, E, k, H, I = 6, 16, 4, 128, 64
    _, gu = make_weight(3, E, 2 * I, H, BF16, 0)
    _, dn = make_weight(4, E, H, I, BF16, 32)
    _, lw = make_weight(5, E, 40, H, BF16, 128)
    x, logits = rand(1, n, H).cuda(), rand(2, n, E, dtype=F32).cuda()
    r = Router(k, "sigmoid", num_groups=4, top_groups=2)

    def step():
        ids, w = route(logits, r)
        return moe_layer(x, gu, dn, ids, w), moe_layer(x, gu, dn, router_logits=logits, router=r), \
            expert_linear(x, lw, ids[:, 0].contiguous())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        x.copy_(rand(20 + i, n, H))
        logits.copy_(rand(30 + i, n, E, dtype=F32))
        g.replay()
        torch.cuda.synchronize()
        want = step()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dtype,g", [(BF16, 0), (F16, 128)])
def test_many_tokens_in_place_strides_and_neighbours(dtype, g):
    """More than 2048 tokens, many to an expert: out is hidden, a row repeated
    by stride 0, a workspace of exactly its size; what lies between and behind
    the rows stays as it was."""
    n, E, k, H, I, offset = 2100, 6, 3, 70, 600, 2
    rg, gu = make_weight(3, E, 2 * I, H, dtype, g)
    rd, dn = make_weight(4, E, H, I, dtype, g)
    ids = make_ids(2, n, E, k, offset, 4)
    w = rand(4, n, k, dtype=F32).abs()
    x = rand(1, n, H, dtype=dtype)
    want, tol = ref.layer(x, rg, rd, ids, w, offset, dtype, dtype)
    nbytes = pkg.moe_layer_workspace_bytes(n, k, E, H, I, group_size=g)
    ws = torch.full((nbytes + 256,), 173, dtype=torch.uint8, device="cuda")
    wide = torch.full((n + 2, H + 9), 7.0, dtype=dtype, device="cuda")
    rows = wide[:n, 3:3 + H]
    rows.copy_(x)
    y = moe_layer(rows, gu, dn, ids.cuda(), w.cuda(), expert_offset=offset, out=rows, workspace=ws[:nbytes])
    close(y, want, tol, "in place")
    wide[:n, 3:3 + H] = 7.0
    assert (wide == 7.0).all() and (ws[nbytes:] == 173).all()
    one = x[:1].cuda().expand(n, H)
    want, tol = ref.layer(x[:1].expand(n, H), rg, rd, ids, w, offset, dtype, F32)
    got = moe_layer(one, gu, dn, ids.cuda(), w.cuda(), expert_offset=offset, out_dtype=F32)
    close(got, want, tol, "repeated row")
    first = ids[:, 0].contiguous()
    out = torch.full((n + 1, 2 * I + 5), 7.0, dtype=dtype, device="cuda")
    y, ytol = ref.linear(x, rg, first, offset, dtype)
    close(expert_linear(x.cuda(), gu, first.cuda(), expert_offset=offset, out=out[:n, 1:1 + 2 * I]), y, ytol, "linear")
    out[:n, 1:1 + 2 * I] = 7.0
    assert (out == 7.0).all()


def test_graph_replays_of_many_tokens():
    """A captured layer and linear product of many tokens to an expert, replayed
    with other ids (experts that had tokens have none, and back), against
    eager calls on another stream at the same time."""
    n, E, k, H, I = 300, 8, 4, 64, 1100
    _, gu = make_weight(3, E, 2 * I, H, BF16, 64)
    _, dn = make_weight(4, E, H, I, BF16, 64)
    x, ids, w = rand(1, n, H).cuda(), make_ids(2, n, E, k).cuda(), rand(3, n, k, dtype=F32).cuda()
    first = ids[:, 0].contiguous()

    def step():
        return moe_layer(x, gu, dn, ids, w), expert_linear(x, gu, first)

    step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        x.copy_(rand(10 + i, n, H))
        ids.copy_(make_ids(20 + i, n, E, k) if i % 2 else torch.full((n, k), i + 1, dtype=torch.int32))
        first.copy_(ids[:, 0])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            eager = step()
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(captured, eager):
            assert torch.equal(a, b) and not b.isnan().any()
        for b in eager:
            b.record_stream(torch.cuda.current_stream())


# -- the operators as a decode step uses them ----------------------------------

@pytest.mark.parametrize("tokens,g", [((3, 0, 5, 1), 0), ((16, 16, 16, 16), 64)])
def test_decode_step_through_dispatch_and_combine(tokens, g):
    """route -> dispatch -> each rank's experts on the rows it received,
    written into its combine buffer -> combine, against the layer's definition
    over all experts; and moe_layer on all tokens at once."""
    ep, E, k, H, I, cap = 4, 16, 4, 96, 48, 16
    rg, gu = make_weight(3, E, 2 * I, H, BF16, g)
    rd, dn = make_weight(4, E, H, I, BF16, g)
    hidden = [rand(s + 1, t, H) for s, t in enumerate(tokens)]
    logits = [rand(s + 11, t, E, dtype=F32) for s, t in enumerate(tokens)]
    r = Router(k, "sigmoid", rand(5, E, dtype=F32, std=0.1).cuda(), num_groups=4, top_groups=3, scale=2.0)
    moe = MoEEp(ep, E, k, cap, H)
    try:
        routed = [route(l.cuda(), r) for l in logits]
        res = moe.dispatch([h.cuda() for h in hidden], [i for i, _ in routed], [w for _, w in routed])
        per = E // ep

        def part(w, d):
            if isinstance(w, torch.Tensor):
                return w[d * per:(d + 1) * per]
            return W4Weights(w.data[d * per:(d + 1) * per], w.scales[d * per:(d + 1) * per], w.rows, w.cols)

        bufs = []
        for d in range(ep):
            buf = moe.get_combine_input_buffer(d, BF16)
            moe_layer(res[d].hidden, part(gu, d), part(dn, d), res[d].topk_ids, res[d].topk_weights,
                      expert_offset=d * per, out=buf)
            bufs.append(buf)
        out = moe.combine(bufs)
        for s in range(ep):
            ids, w = routed[s][0].cpu(), routed[s][1].cpu()
            want, tol = ref.layer(hidden[s], rg, rd, ids, w, 0, BF16, BF16)
            close(moe_layer(hidden[s].cuda(), gu, dn, *routed[s]), want, tol, f"rank {s} at once")
            # each rank's part is rounded to bfloat16 before combine adds them in float32
            parts = torch.zeros_like(want)
            for d in range(ep):
                mine = torch.where(ids // per == d, ids, torch.full_like(ids, -1))
                part_y, part_tol = ref.layer(hidden[s], rg, rd, mine, w, 0, BF16, BF16)
                parts += part_tol + 4 * 2.0 ** -24 * part_y.abs()
            close(out[s], want, ref.rounded(want, parts, BF16), f"rank {s} through dispatch")
    finally:
        moe.destroy()


def by_rank(w, ep):
    """A layer's weights cut into the ranks' experts."""
    if isinstance(w, torch.Tensor):
        return list(w.chunk(ep))
    return [W4Weights(d, s, w.rows, w.cols) for d, s in zip(w.data.chunk(ep), w.scales.chunk(ep))]


@pytest.mark.parametrize("dtype,out_dtype,g", [(BF16, BF16, 0), (F16, F32, 32)])
def test_experts_between_dispatch_and_combine(dtype, out_dtype, g):
    """MoEEp.experts on a step with ranks of unequal and no tokens: the same
    bits as moe_layer rank by rank, the layer's definition after combine, and
    a captured step replayed with other tokens."""
    ep, E, k, H, I, cap = 4, 8, 3, 64, 40, 12
    tokens = (5, 0, 12, 1)
    rg, gu = make_weight(3, E, 2 * I, H, dtype, g)
    rd, dn = make_weight(4, E, H, I, dtype, g)
    gus, dns = by_rank(gu, ep), by_rank(dn, ep)
    r = Router(k, renormalize=False)
    hidden = [rand(s + 1, t, H, dtype=dtype).cuda() for s, t in enumerate(tokens)]
    logits = [rand(s + 11, t, E, dtype=F32).cuda() for s, t in enumerate(tokens)]
    moe = MoEEp(ep, E, k, cap, H, combine_max_elem_bytes=4)
    try:
        def step():
            routed = [route(l, r) for l in logits]
            res = moe.dispatch(hidden, [i for i, _ in routed], [w for _, w in routed])
            bufs = moe.experts(res, gus, dns, dtype=out_dtype)
            return routed, res, bufs, moe.combine(bufs)

        routed, res, bufs, out = step()
        for s in range(ep):
            ids, w = (t.cpu() for t in routed[s])
            want, parts = torch.zeros(2, tokens[s], H, dtype=torch.float64)
            for d in range(ep):      # each rank's part is rounded to out_dtype, then added in float32
                mine = torch.where(ids // (E // ep) == d, ids, torch.full_like(ids, -1))
                y, tol = ref.layer(hidden[s].cpu(), rg, rd, mine, w, 0, dtype, out_dtype)
                want += y
                parts += tol + ep * 2.0 ** -24 * y.abs()
            close(out[s], want, ref.rounded(want, parts, out_dtype), f"rank {s}")
        res = moe.dispatch(hidden, [i for i, _ in routed], [w for _, w in routed])
        bufs = [b.clone() for b in moe.experts(res, gus, dns, dtype=out_dtype)]
        for d in range(ep):
            alone = moe_layer(res[d].hidden, gus[d], dns[d], res[d].topk_ids, res[d].topk_weights,
                              expert_offset=d * (E // ep), out_dtype=out_dtype)
            assert torch.equal(alone, bufs[d])
        for bad in ((res[:3], gus, dns), (res, gus[:3], dns), (res, [gu] * ep, dns), (res, gus, [dn] * ep)):
            with pytest.raises(ValueError):
                moe.experts(*bad)
        moe.combine(bufs)
        with pytest.raises(pkg.MoeEpError):      # no dispatch to follow
            moe.experts(res, gus, dns)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()[3]
        for i in range(4):
            for s in range(ep):
                hidden[s].copy_(rand(40 + 10 * i + s, tokens[s], H, dtype=dtype))
                logits[s].copy_(rand(41 + 20 * i + s, tokens[s], E, dtype=F32))
            graph.replay()
            got = [o.clone() for o in captured]
            torch.cuda.synchronize()
            for a, b in zip(got, step()[3]):
                assert torch.equal(a, b)
    finally:
        moe.destroy()


# -- refusals that need tensors ------------------------------------------------

def test_refusals():
    x = rand(1, 4, 64).cuda()
    w = rand(2, 2, 32, 64).cuda()
    _, w4 = make_weight(3, 2, 32, 64, F16, 32)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: expert_linear(x.float(), w), lambda: expert_linear(x, w.half()),
                lambda: expert_linear(x, w4), lambda: expert_linear(x[:, ::2], w),
                lambda: expert_linear(x[:, :32], w), lambda: expert_linear(x, w, ids[:3]),
                lambda: expert_linear(x, w, ids.float()), lambda: expert_linear(x, w, ids.cpu()),
                lambda: expert_linear(x.cpu(), w), lambda: expert_linear(x, w.cpu()),
                lambda: expert_linear(x, w, out_dtype=F16), lambda: expert_linear(x, w, out=x),
                lambda: expert_linear(x, w.transpose(1, 2)),
                lambda: expert_linear(x, W4Weights(w4.data, w4.scales.bfloat16()[:, :, :3], 32, 64))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: expert_linear(x, w, ids, expert_offset=2 ** 32), lambda: expert_linear(x, w, expert_offset=-1),
                lambda: moe_layer(x, w, rand(4, 2, 64, 16).cuda(), ids.view(4, 1), expert_offset=2 ** 32),
                lambda: route(torch.zeros(1, 4, device="cuda").expand(2 ** 32, 4), Router(1))):
        with pytest.raises(ValueError, match="not in"):
            bad()
    wide = torch.zeros(4, 96, dtype=BF16, device="cuda")
    with pytest.raises(pkg.MoeEpError, match="overlap"):
        expert_linear(wide[:, :64], w, out=wide[:, 40:72])
    dn = rand(4, 2, 64, 16).cuda()
    ids2 = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    logits = torch.zeros(4, 2, device="cuda")
    for bad in (lambda: moe_layer(x, w, dn), lambda: moe_layer(x, w, w, ids2),
                lambda: moe_layer(x, w, dn, ids2, torch.zeros(4, 3, device="cuda")),
                lambda: moe_layer(x, w, dn, ids2, router=Router(2)),
                lambda: moe_layer(x, w, dn, ids2, router_logits=logits),
                lambda: moe_layer(x, w, dn, router_logits=logits[:3], router=Router(2)),
                lambda: moe_layer(x, w, dn, ids2[0]),
                lambda: moe_layer(x, w, dn, ids2, workspace=torch.zeros(64, device="cuda")),
                lambda: route(logits, Router(2, "relu")), lambda: route(logits, Router(2, scale=math.nan)),
                lambda: route(logits, Router(2, bias=torch.zeros(3, device="cuda"))),
                lambda: route(logits.t(), Router(2)), lambda: route(logits.cpu(), Router(2))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: route(logits, Router(3)), lambda: route(logits, Router(2, num_groups=2)),
                lambda: moe_layer(x, w, dn, ids2, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(pkg.MoeEpError):
            bad()
