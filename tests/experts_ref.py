"""Plain float64 forms of the expert-side operators, with the error that
float32 sums and the documented roundings may add, for the GPU tests.

Everything runs on the CPU and shares no code with the package.  Error bounds
count half steps (eps / 2 of a type: bfloat16 2^-8, float16 2^-11, float32
2^-24) and are stated where they are used.
"""

from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# Smallest positive step of a type, halved: what rounding may cost near zero.
HALF_TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def route(logits, top_k, score="softmax", bias=None, num_groups=1, top_groups=1, group_top=2, renormalize=True,
          scale=1.0, invalid=-1):
    """(ids list, weights float64 list) from the definition, one token at a time."""
    big = torch.finfo(torch.float32).max
    x = logits.double().tolist()
    b = None if bias is None else bias.double().tolist()
    E = logits.shape[1]
    ids, ws = [], []
    for row in x:
        row = [min(v, big) if v == v else -math.inf for v in row]
        live = [row[e] > -math.inf and (b is None or b[e] > -math.inf) for e in range(E)]
        if score == "softmax":
            top = max(row)
            p = [math.exp(v - top) if v > -math.inf else 0.0 for v in row]
            z = math.fsum(p)
            p = [v / z if z else 0.0 for v in p]
        else:
            p = [0.0 if v < -700 else 1.0 / (1.0 + math.exp(-v)) for v in row]
        if b is not None:
            key = [p[e] + b[e] if live[e] else -math.inf for e in range(E)]
        else:
            key = p if num_groups > 1 else row
        open_ = [e for e in range(E) if live[e]]
        if num_groups > 1:
            size = E // num_groups
            value = []
            for g in range(num_groups):
                best = sorted((key[e] for e in open_ if e // size == g), reverse=True)[:group_top]
                value.append(sum(best) if best else -math.inf)
            kept = sorted(range(num_groups), key=lambda g: (-value[g], g))[:top_groups]
            open_ = [e for e in open_ if e // size in kept]
        chosen = sorted(open_, key=lambda e: (-key[e], e))[:top_k]
        w = [p[e] for e in chosen]
        z = math.fsum(w) if renormalize else 1.0
        w = [v / z * scale if z > 0 else 0.0 for v in w]
        pad = top_k - len(chosen)
        ids.append(chosen + [invalid] * pad)
        ws.append(w + [0.0] * pad)
    return ids, ws


class W4:
    """4-bit weights as plain integers and scales.  ``expert`` gives the
    matrix and the size its terms may have on the way: the kernels sum q x and
    -8 x apart, so a term is at most (q + 8) |s| |x|."""

    def __init__(self, q, scales, g):
        self.q, self.scales, self.g = q, scales, g
        self.shape = q.shape

    def expert(self, e):
        K = self.q.shape[2]
        s = self.scales[e].double().repeat_interleave(self.g, 1)[:, :K]
        q = self.q[e].double()
        return (q - 8) * s, (q + 8) * s.abs()


class Dense:
    def __init__(self, w):
        self.w = w
        self.shape = w.shape

    def expert(self, e):
        w = self.w[e].double()
        return w, w.abs()


def product(w, x):
    """(x w^T, its float32 error bound).  The kernels sum K terms in eight
    interleaved parts of matrix instructions of 32 terms each: at most 32
    additions inside an instruction, K / 256 + 1 (and as many for 4-bit
    group sums) between instructions, 8 between the parts.  Each addition and
    each 4-bit scaling is off by at most one step (2^-23) of a partial sum,
    and no partial sum is larger than the sum of the terms' magnitudes."""
    W, mag = w
    y = x @ W.t()
    K = W.shape[1]
    adds = 32 + 2 * (K // 256 + 1) + 8 + 4
    return y, adds * 2.0 ** -23 * (x.abs() @ mag.t())


def rounded(y, tol, dtype):
    """The bound after one rounding to dtype."""
    return tol + HALF_STEP[dtype] * (y.abs() + tol) + HALF_TINY[dtype]


def linear(x, weight, ids, offset, out_dtype):
    x = x.double()
    n, N = x.shape[0], weight.shape[1]
    y = torch.zeros(n, N, dtype=torch.float64)
    tol = torch.zeros(n, N, dtype=torch.float64)
    ids = [offset] * n if ids is None else ids.tolist()
    for r, i in enumerate(ids):
        if offset <= i < offset + weight.shape[0]:
            y[r], tol[r] = product(weight.expert(i - offset), x[r])
    return y, rounded(y, tol, out_dtype)


def layer(x, gate_up, down, ids, weights, offset, dtype, out_dtype):
    """The whole layer and its bound.  With d(.) for an error: d(act) =
    1.1 |up| d(gate) + |silu| d(up) (silu's slope is below 1.1) plus 8 float32
    half steps of act for exp and the products, plus the two-part rounding (a
    half step of a half step).  Weighted sums over experts add one rounding
    per expert and wave."""
    x = x.double()
    n, H, inter = x.shape[0], x.shape[1], down.shape[2]
    y = torch.zeros(n, H, dtype=torch.float64)
    tol = torch.zeros(n, H, dtype=torch.float64)
    mag = torch.zeros(n, H, dtype=torch.float64)
    ids = ids.tolist()
    for t in range(n):
        for j, i in enumerate(ids[t]):
            if not offset <= i < offset + gate_up.shape[0]:
                continue
            w = 1.0 if weights is None else float(weights[t, j])
            gu, gt = product(gate_up.expert(i - offset), x[t])
            gate, up, dg, du = gu[:inter], gu[inter:], gt[:inter], gt[inter:]
            silu = gate / (1 + torch.exp(-gate))
            act = silu * up
            da = 1.1 * (up.abs() + du) * dg + silu.abs() * du + 8 * 2.0 ** -24 * act.abs()
            da = da + HALF_STEP[dtype] ** 2 * act.abs() + HALF_TINY[dtype]
            W = down.expert(i - offset)
            v, dv = product(W, act)
            y[t] += w * v
            tol[t] += abs(w) * (dv + da @ W[0].abs().t())
            mag[t] += abs(w) * (act.abs() @ W[1].t())
    tol = tol + (len(ids[0]) + 10) * 2.0 ** -24 * mag if n else tol
    return y, rounded(y, tol, out_dtype)
