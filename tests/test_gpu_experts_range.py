"""The expert-side operators over the range of their numbers: activations from
tiny to large, weights of the routing sums, and real widths, against float64
with bounds that count float32 roundings alone.

Bounds count half steps of float32 (2^-24 of a value)."""

from __future__ import annotations

import math

import pytest
import torch

import combine_token_dest_amd as pkg
from combine_token_dest_amd import MoEEp, Router, W4Weights, expert_linear, moe_layer, route
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, want, tol, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i} got {got[i]}, want {want[i]} "
                             f"+- {tol[i]}")


def is_wide(n, E, k, H, I, g):
    """Whether the library takes its kernels for many tokens: these need room
    for each pair's float32 output beside its activations."""
    return pkg.moe_layer_workspace_bytes(n, k, E, H, I, group_size=g) >= n * k * (6 * -(-I // 16) * 16 + 4 * H)


def powers(seed, shape, lo, hi, dtype):
    """Values of random mantissa and sign, magnitudes 2^lo to 2^(hi + 1)."""
    g = gen(seed)
    m = 1.0 + torch.rand(shape, generator=g)
    e = torch.randint(lo, hi + 1, shape, generator=g).double()
    s = torch.randint(0, 2, shape, generator=g) * 2 - 1
    return (m * s * 2.0 ** e).to(dtype)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("size", ["tiny", "small", "large"])
@pytest.mark.parametrize("g", [0, 32, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_layer_keeps_every_activation_whole(dtype, g, size, many):
    """A token with one element c, gate and up with diagonals: one activation
    v = silu(c a) c b is not zero, so that every sum has a single term and
    nothing hides what happens to v between the products.  v goes from 2^-44
    to above 2^23.

    Half steps: gate and up exact (dense: 22 bits) or one rounding each
    (4 bits), the gate's enlarged by silu's condition 1 + |g (1 - sigmoid)| <= 9
    for g >= -8; exp 4, sum, quotient and product 3: 17.  The down product: v
    in up to six partial products, each but the first added with up to one
    step (2): 10, of the size of q v and 8 v with 4 bits; its scale 1, the
    token's weight 1.  30 in all."""
    n, E, k, H, I = (400 if many else 6), 2, 1, 72, 72
    print(f"[layer range] {dtype} g={g} {size} many={many}", flush=True)
    assert is_wide(n, E, k, H, I, g) == many
    lo_c, hi_c, lo_a, hi_a, lo_b, hi_b = {"tiny": (-10, -8, -11, -9, -11, -9), "small": (-6, -2, -6, -2, -6, -2),
                                          "large": (3, 5, 0, 3, 10, 13)}[size]
    c = powers(1, (n,), lo_c, hi_c, dtype).abs()
    a = powers(2, (E, I), lo_a, hi_a, dtype)
    a = torch.where(a.double() * 2.0 ** (hi_c + 1) < -8, -a, a)
    b = powers(3, (E, I), lo_b, hi_b, dtype)
    x = torch.zeros(n, H, dtype=dtype)
    at = torch.arange(n) * 7 % H
    x[torch.arange(n), at] = c
    ids = (torch.arange(n) % E).to(torch.int32).unsqueeze(1)
    w = torch.rand(n, 1, generator=gen(4)) + 0.5

    def diagonal(v):
        return torch.diag_embed(v)

    std = 2.0 ** -16 if size == "large" else 1.0
    if g == 0:
        gu = torch.cat([diagonal(a), diagonal(b)], 1)
        dn = (torch.randn(E, H, I, generator=gen(5)) * std).to(dtype)
        take_gu, take_dn = gu.cuda(), dn.cuda()
        eff_a, eff_b = a.double(), b.double()
        down, mag = dn.double(), dn.double().abs()
    else:
        # q = 9 on the diagonal: the scale is the value; a group's other elements are zeros
        groups = -(-H // g)
        q = torch.cat([diagonal(torch.ones(E, I)), diagonal(torch.ones(E, I))], 1).to(torch.uint8) + 8
        s = torch.cat([a, b], 1).unsqueeze(2).expand(-1, -1, groups).contiguous()
        take_gu = W4Weights._pack_groups(q.cuda(), s.cuda(), g)
        eff_a, eff_b = a.double(), b.double()
        qd = torch.randint(0, 16, (E, H, I), generator=gen(5), dtype=torch.uint8)
        sd = (torch.randn(E, H, groups, generator=gen(6)) * std).to(dtype)
        take_dn = W4Weights._pack_groups(qd.cuda(), sd.cuda(), g)
        r = ref.W4(qd, sd, g)
        down, mag = (torch.stack(t) for t in zip(*(r.expert(e) for e in range(E))))

    e = ids[:, 0].long()
    gate, up = c.double() * eff_a[e, at], c.double() * eff_b[e, at]
    v = gate / (1 + torch.exp(-gate)) * up
    want = w.double() * down[e, :, at] * v.unsqueeze(1)
    tol = 30 * HALF * w.double() * mag[e, :, at] * v.abs().unsqueeze(1) + 2.0 ** -149
    close(moe_layer(x.cuda(), take_gu, take_dn, ids.cuda(), w.cuda(), out_dtype=F32), want, tol,
          f"activations {v.abs().min():.1e} to {v.abs().max():.1e}")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,E,k", [(1, 1024, 8), (37, 60, 4), (300, 256, 8), (2050, 128, 8), (2100, 256, 16)])
def test_route_weights_are_rounded_once(n, E, k, score, renorm):
    """Each weight is its float64 value rounded to float32: half a step (2^-24),
    and 2^-40 for a float64 sum of up to 1024 exponentials and the quotients.
    Logits of float32 with all their bits, -8 to 8 and a few beyond."""
    print(f"[route weights] n={n} E={E} k={k} {score} renorm={renorm}", flush=True)
    logits = torch.randn(n, E, generator=gen(n + E)) * 3
    logits[:, ::7] *= 2
    r = Router(k, score, renormalize=renorm, scale=2.5)
    ids, w = route(logits.cuda(), r)
    want_ids, want_w = ref.route(logits, k, score, renormalize=renorm, scale=2.5)
    assert ids.tolist() == want_ids
    want = torch.tensor(want_w, dtype=torch.float64)
    close(w, want, want * (HALF + 2.0 ** -40) + 2.0 ** -149, "weights")


def test_int64_ids_past_32_bits_name_no_expert():
    """Ids that an int32 would wrap into the experts' range: zeros, as for any
    other id outside, and no copy of the row in dispatch."""
    E, H, I = 8, 64, 32
    far = [2 ** 32 + 3, -2 ** 32 + 1, 2 ** 40 + 2, -2 ** 63, 2 ** 63 - 1, 2 ** 31, 5, -1]
    n = len(far)
    x = torch.randn(n, H, generator=gen(1)).to(BF16).cuda()
    gu = torch.randn(E, 2 * I, H, generator=gen(2)).to(BF16).cuda()
    dn = torch.randn(E, H, I, generator=gen(3)).to(BF16).cuda()
    ids = torch.tensor(far, device="cuda")
    near = torch.tensor([v if abs(v) < 2 ** 31 else -1 for v in far], dtype=torch.int32, device="cuda")
    assert torch.equal(expert_linear(x, gu, ids), expert_linear(x, gu, near))
    got = moe_layer(x, gu, dn, ids.view(n, 1))
    assert torch.equal(got, moe_layer(x, gu, dn, near.view(n, 1)))
    assert (got[:6] == 0).all() and (got[6] != 0).any()
    moe = MoEEp(1, E, 1, n, H)
    try:
        res = moe.dispatch([x], [ids.view(n, 1)], [torch.ones(n, 1, device="cuda")])
        took = (res[0].topk_ids >= 0) & (res[0].topk_ids < E)
        assert took.flatten().tolist() == [v == 5 for v in far]
        moe.combine([res[0].hidden])
    finally:
        moe.destroy()
