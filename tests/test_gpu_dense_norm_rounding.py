"""rms_norm's 8-bit values are the nearest e4m3 to the quotients, every one of
them: against quotients of whole float64 products, and at values a float32
rounding away from the middles between two e4m3 values."""

from __future__ import annotations

import pytest
import torch

from combine_token_dest_amd import rms_norm
from tests import dense_ref as ref
from tests.test_gpu_experts import rand

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def nearest(x, w, residual, g):
    """The e4m3 values (float64) of 448 s w / max|s w|: s is float32's sum, the
    products and 448 times them are whole in float64, and so is a quotient
    that lies in a middle."""
    s = x.float()
    if residual is not None:
        s = s + residual.float()
    p = s.double() * w.double()
    out = torch.empty_like(p)
    for part in ref.groups_of(x.shape[1], g):
        q = 448.0 * p[:, part] / p[:, part].abs().amax(1, keepdim=True)
        step = 2 * ref.e4m3_half_step(q)
        out[:, part] = torch.round(q / step) * step
    return out


def check(x, w, residual=None, g=0):
    r = rms_norm(x.cuda(), w.cuda(), None if residual is None else residual.cuda(), out_dtype=E4M3, group_size=g)
    got, want = r.rows.cpu().double(), nearest(x, w, residual, g)
    assert int((got != want).sum()) == 0


@pytest.mark.parametrize("g", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,H,weight,residual", [(2000, 4001, F32, False), (1500, 7168, None, True), (3, 1000, F32, True),
                                                 (300, 20000, F32, False), (100, 40003, F32, True), (1, 8, F32, False)])
def test_every_value_is_the_nearest(n, H, weight, residual, dtype, g):
    x = rand(n + H, n, H, dtype=dtype, std=2.0)
    res = rand(n + H + 1, n, H, dtype=dtype, std=3.0) if residual else None
    w = 1 + 0.2 * rand(7, H, dtype=F32)
    check(x, w if weight else w.to(dtype), res, g)


@pytest.mark.parametrize("g", [0, 32, 128])
@pytest.mark.parametrize("H", [128, 2051, 9000, 36000])
def test_values_next_to_the_middles(H, g):
    """Rows of ones, so that the products are the weights: middles between e4m3
    values times an odd k of 20 bits, and float32's neighbours on both sides."""
    t = torch.tensor([17.0, 19, 21, 23, 25, 27, 29, 31], dtype=torch.float64)
    t = torch.cat([t * 2.0 ** e for e in (-10, -6, -3, -1, 0, 3)] + [torch.arange(1, 16, 2) * 2.0 ** -10])
    k = 1048573.0                                          # 5 bits times 20: one rounding to float32 at most
    w = (t * k).to(F32)
    w = torch.cat([w, torch.nextafter(w, torch.tensor(0.0)), torch.nextafter(w, torch.tensor(1e30))])
    w = torch.cat([w, -w])[torch.arange(H) * 7 % (6 * len(t))]
    w[::32] = 448.0 * k
    x = torch.ones(3, H, dtype=BF16)
    x[1] = -0.5
    x[2] = 96
    check(x, w, None, g)
    check(x, torch.flip(w, (0,)), x, g)


@pytest.mark.parametrize("g", [0, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_largest_products_that_float32_does_not_tell_apart(dtype, g):
    """Several products that round to one float32: the quotients are of the largest."""
    H = 1024
    big = torch.tensor([1.0 + 2.0 ** -7, 1.0 + 3 * 2.0 ** -7, 1.0 + 5 * 2.0 ** -7])
    x = torch.full((4, H), 0.25, dtype=dtype)
    w = torch.empty(H)
    for c in range(0, H, 128):
        x[:, c:c + 3] = big.to(dtype)
        # three weights whose products with those are 448 (1 + 2^-24), 448 and 448 (1 - 2^-25), nearly
        w[c:c + 3] = (448.0 * torch.tensor([1 + 2.0 ** -24, 1.0, 1 - 2.0 ** -25], dtype=torch.float64) / big.double()).to(F32)
    t = torch.tensor([17.0, 19, 21, 23, 25, 27, 29, 31]).repeat(H // 8) * 4
    t = torch.stack([t, torch.nextafter(t, torch.tensor(0.0)), torch.nextafter(t, torch.tensor(1e9))], 1).reshape(-1)[:H]
    mask = torch.arange(H) % 128 >= 3
    w[mask] = t[mask]
    check(x, w, None, g)
    check(x[:, torch.arange(H - 1, -1, -1)].contiguous(), torch.flip(w, (0,)), None, g)
