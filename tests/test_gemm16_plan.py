"""How the 16-bit products by expert are cut (csrc/gemm16_plan.hpp, plain C++, compiled here for the host): what it picks
over the range that the calls allow, that its parts fit the workspace that was asked for, and that the sizes of the GPU
tests reach every kernel that any size reaches.  CPU only."""
from __future__ import annotations

import collections
import math
import os
import random
import shutil
import subprocess

import pytest

import q4_swiglu_mlp_amd as Z
from tests.test_gpu_rows16 import CUTS, LARGE, SIZES, WITH_WORKSPACE

CSRC = os.path.join(os.path.dirname(Z.__file__), "csrc")
PROGRAM = r"""
#include <cstdio>
#include "gemm16_plan.hpp"
using namespace zinc;
int main() {
  int M, E, N, K;
  while (std::scanf("%d %d %d %d", &M, &E, &N, &K) == 4) {
    for (Product f : {kForward, kInput, kWeight}) {
      const Gemm16Plan p = plan_gemm16(f, M, E, N, K);
      std::printf("%d %d %d %zu %zu ", p.shape, p.splits, (int)p.queue, p.part, gemm16_part_bytes(f, M, E, N, K));
    }
    const BackwardPlan b = plan_backward(M, E, N, K);
    std::printf("%d %d\n", (int)b.together, (int)b.beside);
  }
}
"""
Cut = collections.namedtuple("Cut", "shape splits queue part room")
PRODUCTS = "c", "da", "dw"


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(at / "plan.cpp"), "-o", str(at / "plan")],
                   check=True)

    def run(sizes):
        """Of each (rows, experts, N, K): the cuts of c, da and dw, and how both gradients are launched."""
        out = subprocess.run([str(at / "plan")], input="".join("%d %d %d %d\n" % s for s in sizes), check=True,
                             stdout=subprocess.PIPE, text=True).stdout.splitlines()
        assert len(out) == len(sizes)
        for line in out:
            v = [int(x) for x in line.split()]
            yield [Cut(*v[5 * i:5 * i + 5]) for i in range(3)], "together" if v[15] else "beside" if v[16] else "apart"

    return run


def drawn(count, seed=1):
    """Sizes over what the calls allow, as far as a card's memory holds the matrices."""
    rng = random.Random(seed)
    log = lambda lo, hi: round(math.exp(rng.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    sizes = []
    while len(sizes) < count:
        rows, E, N, K = log(1, 1 << 20), rng.choice([1, 1, 2, 3, 7, 8, 16, 60, 64, 128, 300, 1024]), 8 * log(1, 8192), 8 * log(1, 8192)
        if 2 * (rows * (N + K) + 2 * E * N * K) < 1 << 37:
            sizes.append((rows, E, N, K))
    return sizes


def kernels(plans):
    """(product, tile, one part | parts | dealt out) that are reached, and the launches of both gradients."""
    found = set()
    for cuts, both in plans:
        for name, c in zip(PRODUCTS, cuts):
            found.add((name, c.shape, "parts" if c.splits > 1 else "queue" if c.queue else "one"))
        found.add(both)
    return found


def test_parts_fit_the_workspace(plan):
    sizes = drawn(20000) + SIZES + LARGE + CUTS + WITH_WORKSPACE
    for (rows, E, N, K), (cuts, both) in zip(sizes, plan(sizes)):
        for name, c, out in zip(PRODUCTS, cuts, (rows * N, rows * K, E * N * K)):
            assert 0 <= c.shape < 4 and 1 <= c.splits <= 16 and not (c.queue and c.splits > 1)
            if c.splits > 1:
                assert c.part >= out and 4 * c.splits * c.part <= c.room, (name, rows, E, N, K)
            assert c.room <= 1 << 26
        assert both != "together" or all(c.queue and c.shape == 0 for c in cuts[1:])
        ask = Z.moe_gemm_workspace_size(rows, E, N, K), Z.moe_gemm_backward_workspace_size(rows, E, N, K)
        assert ask[0] >= cuts[0].room + 1024 and ask[1] >= max(c.room for c in cuts[1:]) + 2048


def test_the_gpu_tests_sizes_reach_every_kernel(plan):
    """Wherever the constants of the cut's model move: what 40000 sizes reach, the tests' lists reach."""
    reached = kernels(plan(SIZES + LARGE + CUTS))
    any_size = kernels(plan(drawn(40000)))
    assert {"together", "beside", "apart"} <= reached
    assert not any_size - reached, sorted(any_size - reached, key=str)


def test_graphs_that_share_a_workspace_use_it(plan):
    """Parts and queues of c, parts and queues of each gradient, and both gradients in one launch."""
    reached = kernels(plan(WITH_WORKSPACE))
    kinds = {(k[0], k[2]) for k in reached if isinstance(k, tuple)}
    assert {(p, how) for p in PRODUCTS for how in ("parts", "queue")} <= kinds and "together" in reached
