"""GPU tests of the adapters and of SwiGLU's gradients where the numbers leave no room: sums that are exact in fp32, so
that any order of them gives the same; factors at opposite ends of fp32's range; scales that nobody has written."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.rows16 as R
import q4_swiglu_mlp_amd as Z
from tests.gpu_common import DEV, dev
from tests.test_gpu_rows16 import GLU, GLU_GATE, HALF, TYPES, close, host, normal, plan_of

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- adapters: A x and dh keep fp32's bits
# rows, adapters, rank, K, N: each number of rank tiles, few and many rows of an adapter, columns in one part and more
EXACT = [(1, 1, 8, 24, 8), (40, 2, 16, 520, 1032), (64, 1, 24, 264, 520), (64, 8, 64, 512, 264), (300, 3, 64, 264, 136),
         (300, 3, 72, 264, 136), (40, 4, 128, 136, 264), (130, 2, 128, 256, 136), (150, 2, 256, 136, 264)]


def digits(rng, ids, cols):
    """Rows whose sum is a 19-bit integer of units of 2^-14 in three values, each exact in 16 bits: one adapter's share the
    first two, of 5 and 7 bits.  Returns them and the columns of the three."""
    z, at = np.zeros((len(ids), cols)), rng.choice(cols, 3, replace=False)
    for e in np.unique(ids):
        mine = ids == e
        z[mine, at[0]], z[mine, at[1]] = rng.integers(16, 32), rng.integers(65, 128) / 2.0 ** 7
    z[:, at[2]] = rng.integers(1, 128, len(ids)) / 2.0 ** 14
    return z, at


def picks(rng, at, E, rank, cols):
    """[E, rank, cols]: the first two digits of every row, the third of every second or so."""
    w = np.zeros((E, rank, cols))
    w[:, :, at[:2]] = 1
    w[:, :, at[2]] = rng.integers(0, 2, (E, rank))
    return w


def balanced(rng, count, n):
    """[count, n]: in each column as many ones as minus ones, eight in all at most, in random places."""
    w, half = np.zeros((count, n)), min(count // 2, 4)
    for j in range(n):
        at = rng.choice(count, 2 * half, replace=False)
        w[at[:half], j], w[at[half:], j] = 1, -1
    return w


@pytest.mark.parametrize("kind", HALF)
@pytest.mark.parametrize("M,E,rank,K,N", EXACT)
def test_adapters_keep_every_bit_of_fp32(kind, M, E, rank, K, N):
    """h = A x is a 19-bit integer (in units of 2^-14), and a sum of eight or fewer of them times 1 or -1 stays below 2^22: every
    partial sum is exact in fp32 in any order, so the outputs are the exact values, rounded once.  The first 12 bits
    cancel, and what remains is the last 7's: of h to 16 bits nothing would be right.  The same for dh."""
    rng = np.random.default_rng(M + rank + K)
    t = TYPES[kind][0]
    to = lambda v: dev(np.asarray(v, dtype=np.float32)).to(t)  # noqa: E731
    ids = (np.arange(M) % E).astype(np.int32)
    if M > 1:
        ids[rng.integers(0, M, M // 10)] = -1
    plan = plan_of(ids, E)
    cpu_plan = [host(v) for v in plan]
    each = lambda count, n: np.stack([balanced(rng, count, n) for _ in range(E)])  # noqa: E731

    def rows_of(cols):          # per adapter balanced over its rows
        z = np.zeros((M, cols))
        for e in range(E):
            mine = np.flatnonzero(ids == e)
            z[mine] = balanced(rng, len(mine), cols)
        return z

    # y and db: the bits are in x
    x, at = digits(rng, ids, K)
    a, b, dy = picks(rng, at, E, rank, K), each(rank, N).transpose(0, 2, 1), rows_of(N)
    y = Z.zinc_lora(to(x), to(a), to(b), None, *plan)
    assert torch.equal(y, to(R.lora(x, a, b, np.ones(E), cpu_plan, np.zeros((M, N)))))
    db = Z.zinc_lora_backward(to(dy), to(x), to(a), to(b), None, *plan)[2]
    assert torch.equal(db, to(R.lora_backward(dy, x, a, b, np.ones(E), cpu_plan, np.zeros((M, K)))[2]))
    # dx and da: they are in dy
    dy, at = digits(rng, ids, N)
    b, a, x = picks(rng, at, E, rank, N).transpose(0, 2, 1), each(rank, K), rows_of(K)
    dx, da, _ = Z.zinc_lora_backward(to(dy), to(x), to(a), to(b), None, *plan)
    want = R.lora_backward(dy, x, a, b, np.ones(E), cpu_plan, np.zeros((M, K)))
    assert torch.equal(dx, to(want[0])) and torch.equal(da, to(want[1]))
    assert M == 1 or (y.any() and db.any() and dx.any() and da.any())


# ---------------------------------------------------------------- adapters without rows
# one part, several parts of the rows, and M = 0
@pytest.mark.parametrize("kind", HALF)
@pytest.mark.parametrize("M,E,K,N", [(50, 4, 264, 136), (3000, 3, 264, 136), (0, 2, 16, 24)])
def test_a_scale_without_rows_is_not_used(kind, M, E, K, N):
    """Slots of a pool that no row uses, with scales nobody has written: their gradients are zeros."""
    rng = np.random.default_rng(M)
    rank = 16
    ids = (np.arange(M) % (E - 1)).astype(np.int32) + 1          # nobody has adapter 0
    x, dy = normal(rng, M, K, kind=kind), normal(rng, M, N, kind=kind)
    a, b = normal(rng, E, rank, K, kind=kind), normal(rng, E, N, rank, kind=kind)
    plan, ones = plan_of(ids, E), torch.ones(E, device=DEV)
    clean = Z.zinc_lora(x, a, b, ones, *plan), *Z.zinc_lora_backward(dy, x, a, b, ones, *plan)
    for bad in (float("nan"), float("inf")):
        scales = ones.clone()
        scales[0 if M else slice(None)] = bad
        got = Z.zinc_lora(x, a, b, scales, *plan), *Z.zinc_lora_backward(dy, x, a, b, scales, *plan)
        for g, c in zip(got, clean):
            assert torch.equal(g, c)
        assert not got[2][0].any() and not got[3][0].any()


# ---------------------------------------------------------------- SwiGLU's gradients, factors at both ends of the range
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d,u", [(-70, 60), (-99, 119), (-126, 127), (60, -70), (127, -126), (127, 127), (0, 0), (90, 100), (-132, 127),
                                 (127, -132)])
def test_swiglu_gradients_of_factors_at_both_ends(kind, d, u):
    """dh and up so far apart that a product of some of the factors leaves fp32's range where dgate does not."""
    rng = np.random.default_rng(5)
    g = np.concatenate([np.linspace(-340, -20, 1000), np.linspace(-20, 90, 536)]).reshape(12, 128)
    sign = rng.choice([-1.0, 1.0], (2, 12, 128)) * rng.uniform(1, 2 - 2.0 ** -6, (2, 12, 128))
    g, dh, up = (dev(v.astype(np.float32)).to(TYPES[kind][0]) for v in (g, np.ldexp(sign[0], d), np.ldexp(sign[1], u)))
    gh, uh, dhh = host(g), host(up), host(dh)
    want_g, want_u = R.swiglu_backward(dhh, gh, uh)
    size = np.abs(dhh) * np.abs(uh) * R.sigmoid(gh) * (1 + np.abs(gh) * R.sigmoid(-gh))
    dg, du = Z.zinc_swiglu_backward(dh, g, up)
    # where a result is past the type's largest value it is infinite, and not compared; below fp32's smallest normal
    # value there are fewer bits: half the smallest step for each of two roundings there
    most = float(torch.finfo(TYPES[kind][0]).max) * (1 - 2.0 ** -7)
    for got, want, slack in ((dg, want_g, GLU_GATE * size), (du, want_u, GLU * np.abs(want_u))):
        fits = np.abs(want) + slack < most
        assert fits.any() and not np.isnan(host(got)).any()
        over = np.abs(want) - slack > most * (1 + 2.0 ** -6)
        assert np.isinf(host(got)[over]).all()
        close(got.cpu()[torch.from_numpy(fits)], want[fits], slack[fits] + 2.0 ** -149, kind)


@pytest.mark.parametrize("kind", list(TYPES))
def test_swiglu_gradients_of_infinite_gates(kind):
    """NaN where the formula has 0 times infinity: dgate of both, dup of minus infinity."""
    inf = float("inf")
    g = torch.tensor([[inf, -inf, 0, 1] * 2], device=DEV).to(TYPES[kind][0])
    one = torch.ones_like(g)
    dg, du = Z.zinc_swiglu_backward(one, g, one)
    assert dg.isnan().tolist() == [[True, True, False, False] * 2]
    assert du.isnan().tolist() == [[False, True, False, False] * 2] and du[0, 0] == inf
