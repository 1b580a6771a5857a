"""Which kernels the GPU tests' sizes reach, by the library's own rule
(csrc/moe_tile_rule.h, host code), on the CPU: every size of tiles of every
product, through memory and through registers, whole and in parts of k.  A
change of the rule that leaves a kernel without a test fails here."""

from __future__ import annotations

import os
import subprocess

import pytest

from tests import test_gpu_dense_adapter as adapter_tests
from tests import test_gpu_dense_gated as gated_tests
from tests import test_gpu_dense_parts as parts_tests
from tests import test_gpu_dense_tiles as tile_tests

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILES = ["256x256", "256x128", "128x128", "64x64", "32x32"]

MAIN = r'''
#include <stdio.h>
#include "moe_tile_rule.h"
using namespace moe_ep_detail;
int main() {
  long long P, Q, k;
  int direct, narrow;
  while (scanf("%lld %lld %lld %d %d", &P, &Q, &k, &direct, &narrow) == 5)
    printf("%d %d %d\n", (int)tile_size(P, Q, k, direct, narrow), product_parts(P, Q, k), gated_few_rows(P / 2));
}
'''


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """(P, Q, k, direct, narrow) of several products -> [(tiles, parts of k, rows of the kernel for few)]."""
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "combine_token_dest_amd", "csrc"),
                    str(d / "rule.cpp"), "-o", str(d / "rule")], check=True)

    def ask(products):
        text = "".join("%d %d %d %d %d\n" % p for p in products)
        out = subprocess.run([str(d / "rule")], input=text, capture_output=True, text=True, check=True).stdout
        rows = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(rows) == len(products)
        return [(TILES[t], parts, few) for t, parts, few in rows]
    return ask


def sizes(test, names):
    """The values of a parametrised test's arguments `names`."""
    for mark in test.pytestmark:
        if mark.name == "parametrize" and mark.args[0] == names:
            return list(mark.args[1])
    raise AssertionError(f"{test.__name__} has no {names}")


def forwards(rule, shapes):
    got = rule([(2 * I, n, H, H % 8 == 0, True) for n, H, I in shapes])
    return {("few", (n + 15) // 16) if n <= few else (tile, H % 8 == 0)
            for (n, H, I), (tile, _, few) in zip(shapes, got)}


def gradients(rule, shapes, two):
    """Of dx and dgate_up: (tiles, direct, in parts)."""
    dx = [(H, n, 2 * I * two, H % 8 == 0 and I % 4 == 0, False) for n, H, I in shapes]
    dw = [(H, 2 * I, n * two, H % 8 == 0, False) for n, H, I in shapes]
    out = []
    for products in (dx, dw):
        parts = [p for _, p, _ in rule([(P, Q, k // two, d, nr) for P, Q, k, d, nr in products])]
        out.append({(tile, bool(p[3]), tile == "64x64" and n > 1)
                    for p, (tile, _, _), n in zip(products, rule(products), parts)})
    return out


def all_tiles(narrow):
    large = {("256x256", True), ("256x128", True)}
    return large | {(t, d) for t in ["128x128", "64x64"] + ["32x32"] * narrow for d in (True, False)}


GATED = (gated_tests.SIZES + sizes(gated_tests.test_largest_tiles, "n,H,I") +
         sizes(gated_tests.test_every_kind_of_tile, "n,H,I") + tile_tests.GATED)
PARTS = sizes(parts_tests.test_two_parts, "n,H,I")
WANT = {(t, d, False) for t, d in all_tiles(False)} | {("64x64", d, True) for d in (True, False)}


def test_forward(rule):
    assert forwards(rule, GATED) == all_tiles(True) | {("few", i) for i in (1, 2, 3, 4)}


@pytest.mark.parametrize("which", [0, 1])
def test_gradients(rule, which):
    assert gradients(rule, GATED, 1)[which] == WANT


@pytest.mark.parametrize("which", [0, 1])
def test_gradients_of_two_parts(rule, which):
    assert gradients(rule, PARTS, 2)[which] == WANT


def test_adapters(rule):
    shapes = [s for _, s in ((0, (n, N, K)) for n, N, K, *_ in sizes(adapter_tests.test_sizes, "n,N,K,L,R") +
                             sizes(adapter_tests.test_every_kind_of_tile, "n,N,K") + [(4100, 4096, 72)] +
                             tile_tests.ADAPTERS)]
    got = {(tile, K % 8 == 0) for (n, N, K), (tile, _, _) in
           zip(shapes, rule([(N, n, K, K % 8 == 0, True) for n, N, K in shapes])) if n > 64}
    assert got == all_tiles(True)
    assert {(n + 15) // 16 for n, _, _ in shapes if n <= 64} == {1, 2, 3, 4}


def turns(rule, products):
    """The most tiles of k that a workgroup goes through, of each kind."""
    most = {}
    for (P, Q, k, direct, _), (tile, parts, _) in zip(products, rule(products)):
        per = {"256x256": 64, "256x128": 64, "128x128": 128, "64x64": 256, "32x32": 256}[tile]
        if tile == "64x64" and parts > 1:
            continue
        most[tile, bool(direct)] = max(most.get((tile, bool(direct)), 0), -(-k // per))
    return most


def test_many_tiles_of_k(rule):
    """Twenty turns of the loop over tiles of k and more in every kind of the
    large tiles' kernels, of each product."""
    kinds = [("256x256", True), ("256x128", True)]
    fwd = turns(rule, [(2 * I, n, H, H % 8 == 0, True) for n, H, I in GATED])
    dx = turns(rule, [(H, n, 2 * I, H % 8 == 0 and I % 4 == 0, False) for n, H, I in GATED])
    dw = turns(rule, [(H, 2 * I, n, H % 8 == 0, False) for n, H, I in GATED])
    ad = turns(rule, [(N, n, K, K % 8 == 0, True) for n, N, K in tile_tests.ADAPTERS])
    for most in (fwd, dx, dw, ad):
        assert all(most.get(kind, 0) >= 20 for kind in kinds), most


def test_parts_of_k(rule):
    """None without two tiles of k each, and no more sums than there is room for."""
    got = rule([(64, 64, 511, 1, 0), (64, 64, 1023, 1, 0), (64, 64, 1024, 1, 0), (64, 64, 1 << 20, 1, 0),
                (64 * 256, 64, 1 << 20, 1, 0), (64 * 128, 64, 1 << 20, 1, 0), (64, 64, 0, 1, 0)])
    assert [p for _, p, _ in got] == [1, 1, 2, 8, 1, 2, 1]
    for P, Q in ((64 * 16, 64 * 16), (64 * 16, 64 * 8), (64 * 32, 64 * 4)):
        (_, parts, _), = rule([(P, Q, 1 << 20, 1, 0)])
        assert 1 <= parts and parts * P * Q <= 512 * 64 * 64
