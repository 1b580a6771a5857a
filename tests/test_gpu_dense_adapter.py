"""adapter_linear on the GPU against its float64 form (tests/dense_ref.py):
types, ranks and sizes, ids of no adapter, strides, special values, streams
and graphs, and the dense operators one after another in a block."""

from __future__ import annotations

import math

import pytest
import torch

from combine_token_dest_amd import adapter_linear, adapter_linear_workspace_bytes, gated_linear, rms_norm
from tests import dense_ref as ref
from tests.test_gpu_experts import close, gen, rand

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make(n, N, K, L, R, dtype, seed=1):
    x, w = rand(seed, n, K, dtype=dtype), rand(seed + 1, N, K, dtype=dtype, std=1 / math.sqrt(K))
    a = rand(seed + 2, L, R, K, dtype=dtype, std=1 / math.sqrt(K))
    b = rand(seed + 3, L, N, R, dtype=dtype, std=1 / math.sqrt(R))
    ids = torch.randint(-1, L + 1, (n,), generator=gen(seed + 4), dtype=torch.int32)
    scales = torch.rand(L, generator=gen(seed + 5)) + 0.5
    return x, w, a, b, ids, scales


def check(got, x, w, a, b, ids, scales):
    y, tol = ref.adapter(x, w, a, b, ids, scales, got.dtype)
    close(got, y, tol, "y")


def run(x, w, a, b, ids, scales, **kw):
    return adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(),
                          scales=None if scales is None else scales.cuda(), **kw)


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, None), (F16, None), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("n,N,K,L,R", [
    (1, 1, 8, 1, 1), (1, 4096, 512, 8, 16), (2, 100, 64, 3, 5), (7, 33, 1000, 4, 64), (16, 256, 264, 64, 8),
    (17, 130, 136, 2, 33), (48, 512, 256, 40, 64), (64, 96, 520, 5, 128), (65, 257, 72, 1, 16), (200, 136, 100, 6, 17),
    (300, 264, 128, 3, 16), (130, 7, 64, 9, 260)])
def test_sizes(n, N, K, L, R, dtype, out_dtype):
    t = make(n, N, K, L, R, dtype)
    check(run(*t, out_dtype=out_dtype), *t)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,N,K,L,R", [(30, 70, 136, 3, 77), (3, 20, 64, 2, 1000), (50, 33, 72, 7, 65), (10, 40, 80, 4, 1024),
                                       (64, 16, 64, 5, 127), (9, 4100, 64, 3, 129)])
def test_ranks_of_several_parts(n, N, K, L, R, dtype):
    t = make(n, N, K, L, R, dtype)
    check(run(*t), *t)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_prompts_one_after_another(dtype):
    """Runs of rows with one adapter, whose ends fall inside tiles; no scales; int64 ids."""
    x, w, a, b, _, _ = make(700, 264, 192, 4, 16, dtype)
    ids = torch.tensor([2] * 130 + [0] * 1 + [-1] * 200 + [3] * 300 + [2] * 69)
    check(run(x, w, a, b, ids, None), x, w, a, b, ids, None)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,N,K", [(5578, 141, 330), (131, 5492, 328), (1314, 5896, 72), (520, 6573, 136),
                                   (70, 90, 330), (65, 80, 520), (4226, 35, 333), (4232, 33, 328)])
def test_every_kind_of_tile(n, N, K, dtype):
    x, w, a, b, _, scales = make(n, N, K, 4, 20, dtype)
    ids = (torch.arange(n) // 77 % 5 - 1).to(torch.int32)
    check(run(x, w, a, b, ids, scales), x, w, a, b, ids, scales)


def test_largest_tiles():
    x, w, a, b, _, scales = make(4100, 4096, 72, 4, 16, BF16)
    ids = (torch.arange(4100) // 333 % 5 - 1).to(torch.int32)
    check(run(x, w, a, b, ids, scales), x, w, a, b, ids, scales)


@pytest.mark.parametrize("n", [5, 140])
def test_no_adapter_at_all(n):
    """Then it is the shared product."""
    x, w, a, b, _, scales = make(n, 72, 64, 3, 16, BF16)
    for bad in (-1, 3, 2 ** 31 - 1, -2 ** 31, 2 ** 32):
        ids = torch.full((n,), bad, dtype=torch.int64)
        got = run(x, w, a, b, ids, scales)
        check(got, x, w, a, b, ids, scales)
    zero = torch.zeros_like(a)
    ids = torch.zeros(n, dtype=torch.int32)
    assert torch.equal(run(x, w, zero, b, ids, scales), got)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [4, 150])
def test_another_rows_adapter_does_not_reach_a_row(n, dtype):
    """Adapters full of infinities and NaN that only some rows name; a row's
    own infinity stays in it."""
    x, w, a, b, _, _ = make(n, 136, 64, 4, 16, dtype)
    a[1], b[2], b[3, ::2] = math.nan, math.inf, math.nan
    scales = torch.tensor([1.0, 1.0, math.inf, 0.5])
    x[2, 3] = math.inf
    ids = torch.tensor([0, 1, 0, -1] + [0] * (n - 4), dtype=torch.int32)
    if n > 100:
        ids[100], ids[101] = 2, 3
    got = run(x, w, a, b, ids, scales).cpu()
    assert got[1].isnan().all() and not got[2].isfinite().any()
    keep = [r for r in range(n) if r not in (1, 2, 100, 101)]
    check(got[keep], x[keep], w, a, b, ids[keep], scales)


def test_float16_low_values_outside_its_range():
    """lora_a x beyond 65504 and far below 2^-14."""
    x, w, a, b, ids, _ = make(150, 72, 64, 2, 16, F16)
    ids = ids.clamp(0, 1)
    a[0] *= 2.0 ** 13
    x = x * 8
    b[0] *= 2.0 ** -13
    a[1] *= 2.0 ** -10
    scales = torch.tensor([1.0, 2.0 ** -14])
    b[1] *= 256
    for rows in (slice(0, 3), slice(0, 150)):
        t = (x[rows], w * 2.0 ** -10, a, b, ids[rows], scales)
        check(run(*t, out_dtype=F32), *t)


@pytest.mark.parametrize("n", [6, 140])
@pytest.mark.parametrize("shift", [0, 1])
def test_strides_alignment_and_neighbours(n, shift):
    N, K, L, R = 88, 104, 3, 16
    x, w, a, b, ids, scales = make(n, N, K, L, R, BF16)
    xb = torch.full((n, 2 * K), math.nan, dtype=BF16, device="cuda")
    wb = torch.full((N, K + 9), math.nan, dtype=BF16, device="cuda")
    xv, wv = xb[:, shift:shift + K], wb[:, shift:shift + K]
    xv.copy_(x.cuda()), wv.copy_(w.cuda())
    out = torch.full((n + 3, N + 6), 4.0, dtype=BF16, device="cuda")
    ws = torch.empty(adapter_linear_workspace_bytes(n, R), dtype=torch.uint8, device="cuda")
    adapter_linear(xv, wv, a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda(), out=out[:n, shift:shift + N],
                   workspace=ws)
    check(out[:n, shift:shift + N], x, w, a, b, ids, scales)
    assert (out[n:] == 4).all() and (out[:, :shift] == 4).all() and (out[:, shift + N:] == 4).all()
    rep = adapter_linear(xv[:1].expand(n, K), wv, a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    check(rep, x[:1].expand(n, K), w, a, b, ids, scales)


def test_no_rows():
    x, w, a, b, ids, scales = make(4, 16, 64, 2, 8, BF16)
    assert run(x[:0], w, a, b, ids[:0], scales).shape == (0, 16)


def test_many_rows():
    x, w, a, b, _, scales = make(2100, 40, 64, 3, 8, BF16)
    ids = (torch.arange(2100) // 100 % 4 - 1).to(torch.int32)
    check(run(x, w, a, b, ids, scales), x, w, a, b, ids, scales)


@pytest.mark.parametrize("n", [3, 140])
def test_streams_and_graph(n):
    sets = [make(n, 264, 136, 5, 16, BF16, seed=20 * i) for i in range(3)]
    dev = [t.cuda() for t in sets[0]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = adapter_linear(*dev[:5], scales=dev[5])
    s.synchronize()
    check(y, *sets[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = adapter_linear(*dev[:5], scales=dev[5])
    for t in sets:
        for d, h in zip(dev, t):
            d.copy_(h)
        graph.replay()
        torch.cuda.synchronize()
        check(y, *t)
        adapter_linear(*dev[:5])
        torch.cuda.synchronize()


@pytest.mark.parametrize("n", [40, 300])
def test_two_streams_at_once(n):
    sets = [make(n, 264, 136, 5, 16, BF16, seed=40 * i) for i in range(2)]
    dev = [[t.cuda() for t in s] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for d, st in zip(dev, streams):
            with torch.cuda.stream(st):
                got.append(adapter_linear(*d[:5], scales=d[5]))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        check(y, *sets[i % 2])


@pytest.mark.parametrize("n,N,K", [(300, 264, 1000), (700, 500, 264), (2300, 4096, 64), (2048, 2050, 72)])
@pytest.mark.parametrize("R", [3, 16, 72])
def test_an_adapter_of_each_rows_own(n, N, K, R):
    """As many adapters in a tile as there are, at every size of tiles."""
    x, w, a, b, ids, scales = make(n, N, K, 40, R, BF16)
    check(run(x, w, a, b, ids, scales), x, w, a, b, ids, scales)


def test_same_bits_each_time():
    t = [v.cuda() for v in make(200, 264, 1032, 8, 16, BF16)]
    y = adapter_linear(*t[:5], scales=t[5])
    for _ in range(3):
        assert torch.equal(adapter_linear(*t[:5], scales=t[5]), y)


@pytest.mark.parametrize("n", [2, 9, 300])
def test_a_block(n):
    """Norm, gated product and an adapted projection one after another, each
    checked on what it was given."""
    H, I, L, R = 136, 72, 3, 16
    x, res, weight = rand(1, n, H), rand(2, n, H), rand(3, H)
    _, w, a, b, ids, scales = make(n, H, I, L, R, BF16)
    gate_up = rand(4, 2 * I, H, std=1 / math.sqrt(H))
    r = rms_norm(x.cuda(), weight.cuda(), res.cuda())
    y, tol = ref.norm(x, weight, res, 1e-6)
    close(r.rows, y, ref.rounded(y, tol, BF16))
    h = gated_linear(r.rows, gate_up.cuda())
    _, _, want, _, _, th = ref.gated(r.rows.cpu(), gate_up)
    close(h, want, ref.rounded(want, th, BF16))
    out = adapter_linear(h, w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    check(out, h.cpu(), w, a, b, ids, scales)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,N,K,R", [(4, 136, 64, 16), (64, 40, 72, 5), (65, 136, 64, 16), (150, 264, 64, 33), (700, 500, 72, 3),
                                     (2300, 4096, 64, 16)])
def test_infinities_and_nan_of_a_rows_own_adapter(n, N, K, R, dtype):
    """They reach a row's results as the formula says, in few rows and many:
    against low values of one bfloat16, of three, negative ones, infinite ones
    and zeros."""
    x, w, a, b, _, _ = make(n, N, K, 4, R, dtype)
    # low values of adapter 0: 0.5, 1 + 2^-7 and some more bits, 0; of adapter 2, with its scale: -2, 6
    a[0], a[2] = 0, 0
    x[:, :3] = torch.tensor([0.5, 1.0, -3.0], dtype=dtype)
    x[:, 3:].abs_().clamp_min_(0.25)
    a[0, 0, 0], a[0, 1, 1], a[0, 1, 0], a[0, 1, 2] = 1, 1, 2.0 ** -7, -(2.0 ** -8) / 3
    a[2, 0, 1], a[2, 1, 2] = 1, 1
    a[1, 1, 5] = math.inf                      # an infinite low value, beside finite ones
    b[0, 0, 0], b[0, 1, 0], b[0, 2, 1], b[0, 3, 1] = math.inf, -math.inf, math.inf, math.nan
    b[0, 4, 2] = math.inf                      # times 0
    b[0, 5, 0], b[0, 5, 1] = math.inf, -math.inf
    b[1, 6, 1], b[1, 7, 1], b[1, 8, 1] = 0.5, -0.5, 0
    b[2, 9, 1], b[2, 10, 0] = math.inf, -math.inf
    ids = (torch.arange(n) % 5 - 1).to(torch.int32)
    scales = torch.tensor([1.0, 0.75, -2.0, 1.0])
    got = run(x, w, a, b, ids, scales).double().cpu()
    want = x.double() @ w.double().t()
    for i in range(4):
        rows = ids == i
        low = (x[rows].double() @ a[i].double().t()) * float(scales[i])
        want[rows] += low @ b[i].double().t()
    assert want.isinf().any() and want.isnan().any() and want.isfinite().any()
    assert torch.equal(got.isnan(), want.isnan())
    special = want.isinf() & ~want.isnan()
    assert torch.equal(got[special], want[special])
    assert torch.equal(got.isfinite(), want.isfinite())
    # the finite ones: of adapters 0, 2 and 3 without the infinities, which are not in their sums
    fine = [torch.nan_to_num(t.float(), nan=0.0, posinf=0.0, neginf=0.0).to(dtype) for t in (a, b)]
    y, tol = ref.adapter(x, w, *fine, ids, scales, dtype)
    keep = want.isfinite()
    assert ((got - y).abs()[keep] <= tol[keep]).all()
