"""Plain float64 forms of the dense operators, with the error that float32
sums and the documented roundings may add, for the GPU tests.

Everything runs on the CPU and shares no code with the package.  Error bounds
count half steps (eps / 2 of a type: bfloat16 2^-8, float16 2^-11, float32
2^-24, e4m3 2^-4) and are stated where they are used.
"""

from __future__ import annotations

import torch

from tests.experts_ref import HALF_STEP, HALF_TINY

U = 2.0 ** -24                # float32's half step


def rounded(y, tol, dtype):
    """The bound after one rounding to dtype."""
    return tol + HALF_STEP[dtype] * (y.abs() + tol) + HALF_TINY[dtype]


def norm(x, weight, residual, eps):
    """(y, its bound before the output's rounding) of float64 rows.

    The kernel's s is off by one float32 half step, its factor 1 / sqrt(m +
    eps) by the same step of s (m's relative error is twice that of s, the
    root halves it) and by its rounding to float32; then come two products'
    roundings.  Six half steps cover the five."""
    s = x.double()
    if residual is not None:
        s = s + residual.double()
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * weight.double()
    return y, 6 * U * y.abs()


def groups_of(H, g):
    g = g or H
    return [slice(a, min(a + g, H)) for a in range(0, H, g)]


def e4m3_half_step(v):
    """Half the distance between e4m3 values at |v|: 2^(e - 4) in [2^e,
    2^(e+1)), 2^-10 below 2^-6."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 4)


def matmul(a, b):
    """(a b^T, its float32 error bound) of float64 matrices.

    The kernels sum k in matrix instructions of 16 or 32 terms, one after
    another in one accumulator, or shared by up to 16 waves that are added in
    turn: at most 32 additions inside an instruction, k / 16 between them, 16
    between waves.  Each is off by at most one step (2^-23) of a partial sum,
    and none is larger than the sum of the terms' magnitudes."""
    k = a.shape[1]
    return a @ b.t(), (k / 16 + 52) * 2.0 ** -23 * (a.abs() @ b.abs().t())


def sigmoid(g):
    e = torch.exp(-g.abs())
    return torch.where(g >= 0, 1 / (1 + e), e / (1 + e))


def silu_slope(g):
    s = sigmoid(g)
    return s * (1 + g * (1 - s))


def gated(x, w):
    """g, u, h and the bounds of each before rounding.  silu's slope is below
    1.1; exp's argument is off by a half step of 1.45 |g|, and eight more half
    steps cover exp, the quotient and the products; where exp(-g) leaves
    float32 (below -88), h may be 0."""
    x, w = x.double(), w.double()
    inter = w.shape[0] // 2
    gu, t = matmul(x, w)
    g, u, tg, tu = gu[:, :inter], gu[:, inter:], t[:, :inter], t[:, inter:]
    silu = g * sigmoid(g)
    h = silu * u
    th = 1.1 * tg * (u.abs() + tu) + silu.abs() * tu + (8 + 2 * g.abs()) * U * h.abs() + 1e-36 * u.abs()
    return g, u, h, tg, tu, th


def gated_grad(x, w, dh, dtype):
    """(dx, its bound, dw, its bound), rounded results' bounds.

    silu's slope is below 1.1 and its second derivative below 0.51.  d is then rounded to
    dtype (float16: scaled so that its largest is at least 2^14, whose
    smallest step is 2^-24), and the results once more."""
    x, w, dh = x.double(), w.double(), dh.double()
    g, u, _, tg, tu, _ = gated(x, w)
    s1, silu = silu_slope(g), g * sigmoid(g)
    d = torch.cat((dh * u * s1, dh * silu), 1)
    more = (10 + 2 * g.abs()) * U                             # exp and the products, as above
    td = torch.cat((dh.abs() * ((1.1 + more) * tu + 0.51 * (u.abs() + tu) * tg + more * u.abs() * (s1.abs() + 0.2)),
                    dh.abs() * (1.1 * tg + more * silu.abs()) + 1e-36), 1)
    td = rounded(d, td, dtype)
    if dtype == torch.float16:
        td = td + d.abs().max() * 2.0 ** -39
    elif dtype == torch.bfloat16:
        td = td + HALF_TINY[dtype]
    dx, t1 = matmul(d, w.t())
    dw, t2 = matmul(d.t(), x.t())
    t1 = t1 * (1 + 2.0 ** -7) + td @ w.abs()
    t2 = t2 * (1 + 2.0 ** -7) + td.t() @ x.abs()
    return dx, rounded(dx, t1, dtype), dw, rounded(dw, t2, dtype)


def adapter(x, w, a, b, ids, scales, out_dtype):
    """(y, its bound) of the shared product with each row's adapter.  low is
    a float32 sum, times its scale (one rounding), and goes into the second
    product whole; both products' sums are added in float32."""
    x = x.double()
    y, t = matmul(x, w.double())
    for i in set(ids.tolist()) & set(range(a.shape[0])):
        rows = ids == i
        s = 1.0 if scales is None else float(scales[i])
        low, tl = matmul(x[rows], a[i].double())
        tl = (tl + 2 * U * low.abs()) * abs(s)
        v, tv = matmul(low * s, b[i].double())
        y[rows] += v
        t[rows] += 3 * tv + tl @ b[i].double().abs().t() + 2 * U * (y[rows].abs() + v.abs())
    return y, rounded(y, t, out_dtype)
