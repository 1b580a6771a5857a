"""The dense products at sizes that the other tests' tiles leave out: each size
of tiles over many tiles of k, and 64 x 64 through registers forward
(tests/test_dense_tiles.py counts what is reached)."""

from __future__ import annotations

import pytest
import torch

from combine_token_dest_amd import gated_linear
from tests.test_gpu_dense_adapter import check, make as make_adapter, run
from tests.test_gpu_dense_gated import check_forward, check_grads, make

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16

GATED = [(4226, 333, 18), (2051, 2088, 964), (2877, 2872, 1412)]
ADAPTERS = [(2051, 2056, 1288), (2877, 2872, 1288)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,H,I", GATED)
def test_gated(n, H, I, dtype):
    x, w, dh = make(n, H, I, dtype)
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    h = gated_linear(gx, gw)
    check_forward(h.detach(), x, w)
    check_grads(*torch.autograd.grad(h, (gx, gw), dh.cuda()), x, w, dh, dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,N,K", ADAPTERS)
def test_adapters(n, N, K, dtype):
    x, w, a, b, _, scales = make_adapter(n, N, K, 4, 20, dtype)
    ids = (torch.arange(n) // 77 % 5 - 1).to(torch.int32)
    check(run(x, w, a, b, ids, scales), x, w, a, b, ids, scales)
