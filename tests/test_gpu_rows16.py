"""GPU tests of the 16-bit products by expert, SwiGLU and the low-rank adapters against float64 (oracle/rows16.py).

Tolerances.  Products of 16-bit values are exact in fp32; a sum of n terms in fp32 is off by at most about n 2^-24
of the sum of their magnitudes, twice that where matrix instructions cut instead of round: (n + 16) 2^-23.  The
final rounding adds half a step of the output's type (2^-11 fp16, 2^-8 bf16, 2^-24 fp32) of the value, and half the
type's smallest step near zero.

SwiGLU, in units of 2^-24: e^-z is off by 3 (the hardware's power 2, the fma 1), s by 3 + 1 (the sum) + 2 (the
reciprocal) = 6, silu(z) u by 6 + 2 products = 8 (powers of two are exact) and dup by as much.  1 - s = e^-z s is
off by 3 + 6 + 1 = 10, so 1 + z (1 - s) by 10 + 1 of the sum of its terms' magnitudes, and dgate by 6 + 11 + 3
products = 20 of that.

Adapters: A x and dh are sums as above; as operands they are two 16-bit terms, off by (half a step)^2: 2^-16 of a
value in bf16, 2^-22 in fp16 and there, where the lower term is subnormal, 2^-38 of the largest value beside it.
The second sum has two terms for each of its products.
(In bf16 there is a third term now, which makes the operand exact: test_gpu_rows16_edges.py.)
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.fp8 as F
import oracle.rows16 as R
import q4_swiglu_mlp_amd as Z
from tests.gpu_common import DEV, dev

pytestmark = pytest.mark.gpu

TYPES = {"f16": (torch.float16, 2.0 ** -11, 2.0 ** -25), "bf16": (torch.bfloat16, 2.0 ** -8, 2.0 ** -134),
         "f32": (torch.float32, 2.0 ** -24, 2.0 ** -150)}
HALF = ["f16", "bf16"]


def host(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def close(got, want, slack, kind, what=""):
    _, half, tiny = TYPES[kind]
    tol = half * (np.abs(want) + slack) + slack + tiny
    err = np.abs(host(got) - want)
    assert np.all(err <= tol), f"{what}: off by {np.max(err / tol):.3g} times the tolerance"


def normal(rng, *shape, kind, size=1.0):
    return dev((size * rng.standard_normal(shape)).astype(np.float32)).to(TYPES[kind][0])


def activations(rng, rows, cols, kind):
    x = rng.standard_normal((rows, cols)) * np.exp(0.5 * rng.standard_normal((rows, 1)))
    return dev(x.astype(np.float32)).to(TYPES[kind][0])


def ranges(rng, rows, E, outside=True):
    """Ascending offsets of uneven ranges, some empty, with rows before the first and behind the last."""
    first = min(rows // 7, 5) if outside else 0
    last = rows - (min(rows // 9, 3) if outside else 0)
    cuts = np.sort(rng.integers(first, last + 1, size=E - 1))
    if E > 2:
        cuts[E // 2] = cuts[E // 2 - 1]
    return np.concatenate([[first], cuts, [last]]).astype(np.int32)


def sums(n):
    return (n + 16) * 2.0 ** -23


# ---------------------------------------------------------------- products by expert
# rows, experts, N, K: single rows, sizes below a tile and past it in each dimension, every tile by the mean rows of an expert
SIZES = [(1, 1, 8, 8), (5, 3, 24, 40), (64, 64, 136, 256), (130, 2, 264, 520), (100, 1, 128, 64), (333, 2, 200, 72),
         (300, 1, 392, 328), (513, 1, 256, 256), (1500, 3, 264, 1032), (700, 2, 520, 136), (2000, 40, 264, 72),
         (900, 2, 8, 1032), (900, 2, 1032, 8)]


@pytest.mark.parametrize("kind", HALF)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows,E,N,K", SIZES)
def test_product(kind, wide, rows, E, N, K):
    rng = np.random.default_rng(rows + N + K)
    a, w, off = activations(rng, rows, K, kind), normal(rng, E, N, K, kind=kind, size=0.1), ranges(rng, rows, E)
    out = "f32" if wide else kind
    c = torch.full((rows, N), -3.0, dtype=TYPES[out][0], device=DEV)
    got = Z.zinc_moe_gemm(a, w, dev(off), out=c)
    assert got is c
    before = np.full((rows, N), -3.0)
    want = R.moe_gemm(host(a), host(w), off, before)
    size = R.moe_gemm(np.abs(host(a)), np.abs(host(w)), off, 0 * before)
    close(c, want, sums(K) * size, out, "c")
    outside = np.ones(rows, bool)
    outside[off[0]:off[-1]] = False
    assert np.all(host(c)[outside] == -3.0)


@pytest.mark.parametrize("kind", HALF)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows,E,N,K", SIZES)
def test_product_gradients(kind, wide, rows, E, N, K):
    rng = np.random.default_rng(rows + N + K + 1)
    a, w, off = activations(rng, rows, K, kind), normal(rng, E, N, K, kind=kind, size=0.1), ranges(rng, rows, E)
    dc = normal(rng, rows, N, kind=kind)
    out = "f32" if wide else kind
    da = torch.full((rows, K), -3.0, dtype=TYPES[out][0], device=DEV)
    dw = torch.full((E, N, K), -3.0, dtype=TYPES[out][0], device=DEV)
    got = Z.zinc_moe_gemm_backward(dc, a, w, dev(off), da=da, dw=dw)
    assert got[0] is da and got[1] is dw
    before = np.full((rows, K), -3.0)
    want_a, want_w = R.moe_gemm_backward(host(dc), host(a), host(w), off, before)
    size_a, size_w = R.moe_gemm_backward(*(np.abs(host(t)) for t in (dc, a, w)), off, 0 * before)
    close(da, want_a, sums(N) * size_a, out, "da")
    close(dw, want_w, sums(rows) * size_w, out, "dw")
    outside = np.ones(rows, bool)
    outside[off[0]:off[-1]] = False
    assert np.all(host(da)[outside] == -3.0)
    for e in range(E):
        assert off[e] < off[e + 1] or not host(dw[e]).any()
    only_a, none = Z.zinc_moe_gemm_backward(dc, a, w, dev(off), da_dtype=TYPES[out][0], want_dw=False)
    assert none is None and torch.equal(only_a[off[0]:off[-1]], da[off[0]:off[-1]])
    none, only_w = Z.zinc_moe_gemm_backward(dc, a, w, dev(off), dw_dtype=TYPES[out][0], want_da=False)
    assert none is None and torch.equal(only_w, dw)


# many units of the largest tile (dealt out from queues, both gradients in one launch), more experts than XCDs
# and not a multiple of them, many small experts, and few units with a long summed dimension (in parts)
LARGE = [(30000, 20, 1032, 1544), (24000, 3, 2056, 1032), (12000, 1, 3096, 1032), (3000, 1000, 24, 40), (33, 1, 136, 8200),
         (70, 2, 8200, 72), (9000, 1, 72, 136), (20000, 2, 264, 64)]


@pytest.mark.parametrize("kind,wide", [("bf16", False), ("f16", True)])
@pytest.mark.parametrize("rows,E,N,K", LARGE)
def test_products_of_many_and_of_few_units(kind, wide, rows, E, N, K):
    rng = np.random.default_rng(rows + N)
    a, w, off = activations(rng, rows, K, kind), normal(rng, E, N, K, kind=kind, size=0.1), ranges(rng, rows, E)
    dc = normal(rng, rows, N, kind=kind)
    out = "f32" if wide else kind
    t = TYPES[out][0]
    c, da = (torch.full((rows, n), -3.0, dtype=t, device=DEV) for n in (N, K))
    Z.zinc_moe_gemm(a, w, dev(off), out=c)
    _, dw = Z.zinc_moe_gemm_backward(dc, a, w, dev(off), da=da, dw_dtype=t)
    ah, wh, dch = host(a), host(w), host(dc)
    am, wm, dm = np.abs(ah), np.abs(wh), np.abs(dch)
    close(c, R.moe_gemm(ah, wh, off, np.full((rows, N), -3.0)),
          sums(K) * R.moe_gemm(am, wm, off, np.zeros((rows, N))), out, "c")
    want_a, want_w = R.moe_gemm_backward(dch, ah, wh, off, np.full((rows, K), -3.0))
    size_a, size_w = R.moe_gemm_backward(dm, am, wm, off, np.zeros((rows, K)))
    close(da, want_a, sums(N) * size_a, out, "da")
    close(dw, want_w, sums(rows) * size_w, out, "dw")
    alone = Z.zinc_moe_gemm_backward(dc, a, w, dev(off), da_dtype=t, want_dw=False)[0]
    assert torch.equal(alone[off[0]:off[-1]], da[off[0]:off[-1]])
    assert torch.equal(Z.zinc_moe_gemm_backward(dc, a, w, dev(off), dw_dtype=t, want_da=False)[1], dw)
    # the rows in other places of the same call
    for _ in range(2):
        again = torch.full_like(c, -3.0)
        Z.zinc_moe_gemm(a, w, dev(off), out=again)
        assert torch.equal(again, c)


# every tile of c, of da and of dw, in one part, in parts and dealt out from queues; both gradients in one launch, one
# after the other, and side by side
CUTS = [(1, 1, 8, 8), (1, 1, 8, 800), (1, 2, 840, 8), (1685, 2, 8, 8), (33443, 3, 16, 8), (2777, 1, 8, 5856),
        (11334, 1, 1704, 8), (17745, 9, 632, 8), (30758, 60, 152, 8), (34823, 1, 16, 6400), (33078, 9, 904, 8),
        (16867, 20, 136, 240), (8931, 9, 160, 2240), (24545, 130, 192, 304), (4268, 20, 1640, 448), (210, 300, 672, 264),
        (34950, 130, 8, 136), (2008, 1, 3040, 2336), (19076, 1, 8, 920), (636, 300, 912, 144), (9572, 9, 2056, 136),
        (27503, 130, 392, 160), (17469, 130, 984, 288), (229, 130, 288, 928), (77, 130, 728, 144), (13234, 9, 2656, 136),
        (150, 130, 2992, 136), (86, 130, 464, 136), (25271, 9, 1224, 144), (11663, 20, 2120, 136), (713, 300, 80, 8),
        (269, 300, 2616, 8), (169, 300, 8, 6968), (17042, 60, 648, 688), (1, 1, 1264, 8),
        (28194, 130, 200, 376), (3739, 20, 8, 3168), (17984, 130, 312, 688), (1088, 300, 160, 432),
        (3, 1, 65536, 8), (3, 2, 8, 65536), (300, 1, 65536, 72), (300, 1024, 72, 264)]


@pytest.mark.parametrize("kind,wide", [("bf16", True), ("f16", False)])
@pytest.mark.parametrize("rows,E,N,K", CUTS)
def test_every_cut(kind, wide, rows, E, N, K):
    rng = np.random.default_rng(rows + E)
    a, w, off = activations(rng, rows, K, kind), normal(rng, E, N, K, kind=kind, size=0.1), ranges(rng, rows, E)
    dc = normal(rng, rows, N, kind=kind)
    out = "f32" if wide else kind
    t = TYPES[out][0]
    c = torch.full((rows, N), -3.0, dtype=t, device=DEV)
    das = [torch.full((rows, K), -3.0, dtype=t, device=DEV) for _ in range(2)]
    dws = [torch.full((E, N, K), -3.0, dtype=t, device=DEV) for _ in range(2)]
    Z.zinc_moe_gemm(a, w, dev(off), out=c)
    Z.zinc_moe_gemm_backward(dc, a, w, dev(off), da=das[0], dw=dws[0])
    Z.zinc_moe_gemm_backward(dc, a, w, dev(off), da=das[1], want_dw=False)
    Z.zinc_moe_gemm_backward(dc, a, w, dev(off), dw=dws[1], want_da=False)
    ah, wh, dch = host(a), host(w), host(dc)
    am, wm, dm = np.abs(ah), np.abs(wh), np.abs(dch)
    close(c, R.moe_gemm(ah, wh, off, np.full((rows, N), -3.0)),
          sums(K) * R.moe_gemm(am, wm, off, np.zeros((rows, N))), out, "c")
    want_a, want_w = R.moe_gemm_backward(dch, ah, wh, off, np.full((rows, K), -3.0))
    size_a, size_w = R.moe_gemm_backward(dm, am, wm, off, np.zeros((rows, K)))
    for da, dw in zip(das, dws):
        close(da, want_a, sums(N) * size_a, out, "da")
        close(dw, want_w, sums(rows) * size_w, out, "dw")
        for e in range(E):
            assert off[e] < off[e + 1] or not bool(dw[e].any())


@pytest.mark.parametrize("rows,E", [(1, 1), (40, 3), (700, 2), (2000, 3)])
def test_products_keep_nan_in_its_place(rows, E):
    """Rows outside the ranges, other experts' rows and weights, and what lies behind a row's end add nothing."""
    rng = np.random.default_rng(rows)
    N, K, kind = 264, 72, "bf16"
    a, w, dc = activations(rng, rows, K, kind), normal(rng, E, N, K, kind=kind), normal(rng, rows, N, kind=kind)
    off = ranges(rng, rows, E)
    if rows == 1:
        off[:] = [0, 1]
    clean = [host(t) for t in (Z.zinc_moe_gemm(a, w, dev(off), torch.float32),
                               *Z.zinc_moe_gemm_backward(dc, a, w, dev(off), torch.float32, torch.float32))]
    nan = float("nan")
    inside = np.arange(off[0], off[-1])
    hit = int(inside[len(inside) // 2])
    expert = int(np.searchsorted(off, hit, side="right") - 1)
    a2, dc2, w2 = a.clone(), dc.clone(), w.clone()
    for t in (a2, dc2):
        t[:off[0]], t[off[-1]:], t[hit] = nan, nan, nan
    got = [host(t) for t in (Z.zinc_moe_gemm(a2, w, dev(off), torch.float32),
                             *Z.zinc_moe_gemm_backward(dc2, a2, w, dev(off), torch.float32, torch.float32))]
    others = inside[inside != hit]
    for i in (0, 1):
        assert np.array_equal(got[i][others], clean[i][others]) and np.isnan(got[i][hit]).all()
    for e in range(E):
        assert np.isnan(got[2][e]).all() if e == expert else np.array_equal(got[2][e], clean[2][e])
    w2[expert] = nan
    c, da = (host(t) for t in (Z.zinc_moe_gemm(a, w2, dev(off), torch.float32),
                               Z.zinc_moe_gemm_backward(dc, a, w2, dev(off), torch.float32, want_dw=False)[0]))
    mine = (inside >= off[expert]) & (inside < off[expert + 1])
    assert np.isnan(c[inside[mine]]).all() and np.array_equal(c[inside[~mine]], clean[0][inside[~mine]])
    assert np.isnan(da[inside[mine]]).all() and np.array_equal(da[inside[~mine]], clean[1][inside[~mine]])


@pytest.mark.parametrize("rows", [50, 900])
def test_product_offsets_are_cut(rows):
    rng = np.random.default_rng(rows)
    a, w, dc = (normal(rng, *s, kind="f16") for s in ((rows, 72), (3, 40, 72), (rows, 40)))
    off = np.array([np.iinfo(np.int32).min, rows // 2, rows // 2, np.iinfo(np.int32).max], dtype=np.int32)
    want = R.moe_gemm(host(a), host(w), off, np.zeros((rows, 40)))
    size = R.moe_gemm(np.abs(host(a)), np.abs(host(w)), off, np.zeros((rows, 40)))
    close(Z.zinc_moe_gemm(a, w, dev(off)), want, sums(72) * size, "f16")
    da, dw = Z.zinc_moe_gemm_backward(dc, a, w, dev(off))
    want_a, want_w = R.moe_gemm_backward(host(dc), host(a), host(w), off, np.zeros((rows, 72)))
    size_a, size_w = R.moe_gemm_backward(*(np.abs(host(t)) for t in (dc, a, w)), off, np.zeros((rows, 72)))
    close(da, want_a, sums(40) * size_a, "f16")
    close(dw, want_w, sums(rows) * size_w, "f16")


def test_product_without_rows():
    w = torch.ones((3, 16, 24), dtype=torch.float16, device=DEV)
    a, dc = (torch.empty((0, n), dtype=torch.float16, device=DEV) for n in (24, 16))
    off = torch.tensor([0, 0, 5, 9], dtype=torch.int32, device=DEV)
    assert Z.zinc_moe_gemm(a, w, off).shape == (0, 16)
    dw = torch.full((3, 16, 24), 7.0, device=DEV)
    da, _ = Z.zinc_moe_gemm_backward(dc, a, w, off, dw=dw)
    assert da.shape == (0, 24) and not dw.any()
    none = torch.zeros(4, dtype=torch.int32, device=DEV)
    a = torch.full((9, 24), float("nan"), dtype=torch.float16, device=DEV)
    c = torch.full((9, 16), 2.0, dtype=torch.float16, device=DEV)
    Z.zinc_moe_gemm(a, w, none, out=c)
    assert bool((c == 2).all())
    dw.fill_(7.0)
    Z.zinc_moe_gemm_backward(c, a, w, none, dw=dw, want_da=False)
    assert not dw.any()


# ---------------------------------------------------------------- SwiGLU
GLU, GLU_GATE = 8 * 2.0 ** -24, 20 * 2.0 ** -24


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 24), (257, 1032), (2050, 4104)])
def test_swiglu(kind, rows, cols):
    rng = np.random.default_rng(rows)
    g, u, dh = (3.0 * normal(rng, rows, cols, kind=kind) for _ in range(3))
    wide = rng.uniform(-110, 110, size=min(rows * cols, 500))
    g.view(-1)[:len(wide)] = dev(wide.astype(np.float32)).to(g.dtype)
    gh, uh, dhh = host(g), host(u), host(dh)
    want = R.swiglu(gh, uh)
    close(Z.zinc_swiglu(g, u), want, GLU * np.abs(want), kind, "h")
    dg, du = Z.zinc_swiglu_backward(dh, g, u)
    want_g, want_u = R.swiglu_backward(dhh, gh, uh)
    size = np.abs(dhh * uh) * R.sigmoid(gh) * (1 + np.abs(gh) * R.sigmoid(-gh))
    close(dg, want_g, GLU_GATE * size, kind, "dgate")
    close(du, want_u, GLU * np.abs(want_u), kind, "dup")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_swiglu_over_the_types_range(kind):
    """Gates so low that s leaves fp32's range, with factors that bring the products back."""
    g = dev(np.linspace(-260, 260, 1040).astype(np.float32)).to(TYPES[kind][0]).view(5, 208)
    u = torch.full_like(g, 2.0 ** 60)
    dh = torch.full_like(g, 2.0 ** 50)
    gh, uh, dhh = host(g), host(u), host(dh)
    want = R.swiglu(gh, uh)
    least = 2.0 ** -126                        # below it fp32 has fewer bits, or none
    close(Z.zinc_swiglu(g, u), want, GLU * np.abs(want) + least, kind, "h")
    dg, du = Z.zinc_swiglu_backward(dh, g, u)
    want_g, want_u = R.swiglu_backward(dhh, gh, uh)
    size = np.abs(dhh * uh) * R.sigmoid(gh) * (1 + np.abs(gh) * R.sigmoid(-gh))
    close(dg, want_g, GLU_GATE * size + least, kind, "dgate")
    close(du, want_u, GLU * np.abs(want_u) + least, kind, "dup")
    big = torch.tensor([[1e30, -1e30, 3e38, -3e38, 65000.0, -65000.0, 0.0, -0.0]], device=DEV).to(g.dtype)
    one = torch.ones_like(big)
    dg, du = Z.zinc_swiglu_backward(one, big, one)
    assert torch.equal(dg, torch.tensor([[1, 0, 1, 0, 1, 0, 0.5, 0.5]], device=DEV).to(g.dtype))
    assert torch.equal(du, torch.where(big > 0, big, 0)) and torch.equal(Z.zinc_swiglu(big, one), du)


@pytest.mark.parametrize("kind", list(TYPES))
def test_swiglu_not_finite_stays_in_its_place(kind):
    rng = np.random.default_rng(0)
    g, u, dh = (normal(rng, 9, 24, kind=kind) for _ in range(3))
    clean = [Z.zinc_swiglu(g, u), *Z.zinc_swiglu_backward(dh, g, u)]
    at = torch.zeros(9, 24, dtype=torch.bool, device=DEV)
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
        g[i, i], u[3 + i, 5], dh[6 + i, 7] = v, v, v
        at[i, i] = at[3 + i, 5] = at[6 + i, 7] = True
    for got, want in zip([Z.zinc_swiglu(g, u), *Z.zinc_swiglu_backward(dh, g, u)], clean):
        assert torch.equal(got[~at], want[~at])
    h, (dg, du) = Z.zinc_swiglu(g, u), Z.zinc_swiglu_backward(dh, g, u)
    assert bool(h[0, 0].isnan()) and bool(h[3, 5].isnan()) and bool(dg[0, 0].isnan()) and bool(du[0, 0].isnan())
    assert bool(h[1, 1].isinf()) and bool(h[4, 5].isinf()) and bool(h[5, 5].isinf()) and bool(h[2, 2].isnan())


# ---------------------------------------------------------------- adapters
def plan_of(ids, E):
    return Z.zinc_moe_sort(dev(ids.reshape(-1, 1).astype(np.int32)), E)


def adapter_ids(rng, M, E):
    """Runs of rows and single ones, a tenth of the rows without an adapter, and one adapter nobody has."""
    ids = rng.integers(0, E, size=M)
    run = rng.integers(1, 9, size=M)
    ids = np.repeat(ids, run)[:M]
    ids[rng.random(M) < 0.1] = -1
    if E > 1:
        ids[ids == E - 1] = 0
    return ids.astype(np.int32)


LORA = [(1, 1, 8, 8, 8), (1, 4, 16, 264, 72), (7, 3, 8, 40, 520), (33, 64, 24, 136, 1032), (64, 1, 64, 512, 264),
        (200, 2, 16, 1032, 1040), (300, 3, 72, 264, 520), (130, 2, 128, 256, 136), (150, 2, 256, 136, 264),
        (90, 3, 200, 72, 72), (1500, 2, 32, 520, 136), (1100, 1, 40, 72, 600), (3, 1, 256, 65536, 8), (5, 2, 8, 8, 65536),
        (130, 1, 64, 65536, 72), (200, 1024, 16, 72, 40)]


def lora_inputs(rng, M, E, rank, K, N, kind):
    x = activations(rng, M, K, kind)
    a = normal(rng, E, rank, K, kind=kind, size=K ** -0.5)
    b = normal(rng, E, N, rank, kind=kind, size=rank ** -0.5)
    scales = dev(rng.uniform(0.25, 2.0, E).astype(np.float32))
    ids = adapter_ids(rng, M, E)
    return x, a, b, scales, ids, F.sort(ids.reshape(-1, 1), E), plan_of(ids, E)


def split_off(kind):
    return 2.0 ** -16 if kind == "bf16" else 2.0 ** -22


def lora_slack(x, a, b, s, plan, kind):
    """How far the adapters' part of y may be off before its rounding."""
    x, a, b, s = (np.abs(host(t)) for t in (x, a, b, s))
    K, rank = x.shape[1], a.shape[1]
    zero = np.zeros((x.shape[0], b.shape[1]))
    size = R.lora(x, a, b, s, plan, zero)
    slack = (sums(K) + split_off(kind) + sums(2 * rank) + 4 * 2.0 ** -24) * size
    if kind == "f16":      # 2^-38 of the row's largest, for each of its values
        for e in range(len(a)):
            rows = plan[2][plan[0][e]:plan[0][e + 1]]
            if len(rows):
                h = x[rows] @ a[e].T
                slack[rows] += s[e] * 2.0 ** -38 * h.max(1, keepdims=True) * b[e].sum(1)
    return slack


@pytest.mark.parametrize("kind", HALF)
@pytest.mark.parametrize("M,E,rank,K,N", LORA)
def test_lora(kind, M, E, rank, K, N):
    rng = np.random.default_rng(M + rank + K)
    x, a, b, s, ids, plan, gpu_plan = lora_inputs(rng, M, E, rank, K, N, kind)
    base = normal(rng, M, N, kind=kind)
    slack = lora_slack(x, a, b, s, plan, kind)
    size = slack + 2.0 ** -23 * np.abs(host(base))
    want = R.lora(host(x), host(a), host(b), host(s), plan, host(base))
    keep = base.clone()
    y = Z.zinc_lora(x, a, b, s, *gpu_plan, base=base)
    close(y, want, size, kind, "y")
    assert torch.equal(base, keep)
    without = torch.from_numpy(ids < 0).to(DEV)
    assert torch.equal(y[without], base[without])
    again = base.clone()
    assert Z.zinc_lora(x, a, b, s, *gpu_plan, base=again, y=again) is again and torch.equal(again, y)
    alone = Z.zinc_lora(x, a, b, s, *gpu_plan)
    zero = np.zeros((M, N))
    close(alone, R.lora(host(x), host(a), host(b), host(s), plan, zero), slack, kind, "no base")
    assert not alone[without].any()
    ones = Z.zinc_lora(x, a, b, None, *gpu_plan)
    one = torch.ones(E, device=DEV)
    assert torch.equal(ones, Z.zinc_lora(x, a, b, one, *gpu_plan))


@pytest.mark.parametrize("kind", HALF)
@pytest.mark.parametrize("M,E,rank,K,N", LORA)
def test_lora_gradients(kind, M, E, rank, K, N):
    rng = np.random.default_rng(M + rank + K + 1)
    x, a, b, s, ids, plan, gpu_plan = lora_inputs(rng, M, E, rank, K, N, kind)
    base, dy = normal(rng, M, K, kind=kind), normal(rng, M, N, kind=kind)
    da = torch.full((E, rank, K), 5.0, dtype=x.dtype, device=DEV)
    db = torch.full((E, N, rank), 5.0, dtype=x.dtype, device=DEV)
    dx, got_a, got_b = Z.zinc_lora_backward(dy, x, a, b, s, *gpu_plan, base=base, da=da, db=db)
    assert got_a is da and got_b is db
    want = R.lora_backward(*(host(t) for t in (dy, x, a, b, s)), plan, host(base))
    mags = [np.abs(host(t)) for t in (dy, x, a, b, s)]
    size = R.lora_backward(*mags, plan, 0 * host(base))
    most = int(np.diff(plan[0]).max())
    each = split_off(kind) + 4 * 2.0 ** -24
    slack_x = (sums(N) + sums(2 * rank) + each) * size[0] + 2.0 ** -23 * np.abs(host(base))
    slack_a = (sums(N) + sums(2 * most + 64) + each) * size[1]
    slack_b = (sums(K) + sums(2 * most + 64) + each) * size[2]
    if kind == "f16":
        dyh, xh, ah, bh, sh = mags
        for e in range(E):
            rows = plan[2][plan[0][e]:plan[0][e + 1]]
            if len(rows):
                h, dh = xh[rows] @ ah[e].T, dyh[rows] @ bh[e]
                slack_x[rows] += sh[e] * 2.0 ** -38 * dh.max(1, keepdims=True) * ah[e].sum(0)
                slack_a[e] += sh[e] * 2.0 ** -38 * dh.max() * xh[rows].sum(0)
                slack_b[e] += sh[e] * 2.0 ** -38 * h.max() * dyh[rows].sum(0)[:, None]
    close(dx, want[0], slack_x, kind, "dx")
    close(da, want[1], slack_a, kind, "da")
    close(db, want[2], slack_b, kind, "db")
    without = torch.from_numpy(ids < 0).to(DEV)
    assert torch.equal(dx[without], base[without])
    if E > 1:
        assert not da[E - 1].any() and not db[E - 1].any()
    again = base.clone()
    for want_dx, want_da, want_db in ((True, False, False), (False, True, False), (False, False, True)):
        part = Z.zinc_lora_backward(dy, x, a, b, s, *gpu_plan, base=again, dx=again if want_dx else None,
                                    want_dx=want_dx, want_da=want_da, want_db=want_db)
        for p, full, wanted in zip(part, (dx, da, db), (want_dx, want_da, want_db)):
            assert torch.equal(p, full) if wanted else p is None


@pytest.mark.parametrize("M,E", [(1, 1), (50, 4), (400, 2)])
def test_lora_without_any_adapter(M, E):
    rng = np.random.default_rng(M)
    x, base, dy = (normal(rng, M, n, kind="f16") for n in (64, 40, 40))
    a, b = normal(rng, E, 16, 64, kind="f16"), normal(rng, E, 40, 16, kind="f16")
    for wild in (-1, E, np.iinfo(np.int32).max, np.iinfo(np.int32).min):
        plan = plan_of(np.full(M, wild, np.int32), E)
        assert torch.equal(Z.zinc_lora(x, a, b, None, *plan, base=base), base)
        assert not Z.zinc_lora(x, a, b, None, *plan).any()
        dx, da, db = Z.zinc_lora_backward(dy, x, a, b, None, *plan)
        assert not dx.any() and not da.any() and not db.any()


def test_lora_without_rows():
    a, b = torch.ones((2, 8, 16), dtype=torch.float16, device=DEV), torch.ones((2, 24, 8), dtype=torch.float16, device=DEV)
    plan = plan_of(np.zeros(0, np.int32), 2)
    x, dy = (torch.empty((0, n), dtype=torch.float16, device=DEV) for n in (16, 24))
    assert Z.zinc_lora(x, a, b, None, *plan).shape == (0, 24)
    dx, da, db = Z.zinc_lora_backward(dy, x, a, b, None, *plan)
    assert dx.shape == (0, 16) and not da.any() and not db.any()


@pytest.mark.parametrize("M", [20, 500])
def test_lora_keeps_nan_in_its_place(M):
    """A row that is not finite reaches its own y and dx, and its adapter's gradients, and nothing else."""
    rng = np.random.default_rng(M)
    E, kind = 3, "f16"
    x, a, b, s, ids, plan, gpu_plan = lora_inputs(rng, M, E, 24, 72, 136, kind)
    ids = (np.arange(M) % 2).astype(np.int32)
    ids[::5] = -1
    gpu_plan = plan_of(ids, E)
    base, dbase, dy = normal(rng, M, 136, kind=kind), normal(rng, M, 72, kind=kind), normal(rng, M, 136, kind=kind)
    run = lambda x, dy: [Z.zinc_lora(x, a, b, s, *gpu_plan, base=base),  # noqa: E731
                         *Z.zinc_lora_backward(dy, x, a, b, s, *gpu_plan, base=dbase)]
    clean = run(x, dy)
    for bad in (float("nan"), float("inf")):
        x2, dy2 = x.clone(), dy.clone()
        x2[7], dy2[7], x2[5], dy2[5] = bad, bad, bad, bad      # adapter 1; and a row without one
        got = run(x2, dy2)
        others = torch.arange(M, device=DEV) != 7
        for i in (0, 1):
            assert torch.equal(got[i][others], clean[i][others]) and not got[i][7].isfinite().any()
        for i in (2, 3):
            assert torch.equal(got[i][0], clean[i][0]) and not got[i][1].isfinite().any() and not got[i][2].any()


@pytest.mark.parametrize("large", [2.0 ** 9, 2.0 ** -14])
def test_lora_fp16_beyond_its_range_inside(large):
    """A x of up to 2^19, and gradients far below fp16's smallest values, keep their bits until y."""
    rng = np.random.default_rng(3)
    M, E, rank, K, N = 130, 2, 16, 256, 136
    x, a, _, s, ids, plan, gpu_plan = lora_inputs(rng, M, E, rank, K, N, "f16")
    x = x * large
    a = normal(rng, E, rank, K, kind="f16", size=8.0 if large > 1 else 1e-4)
    b = normal(rng, E, N, rank, kind="f16", size=2.0 ** -14 if large > 1 else 64.0)
    y = Z.zinc_lora(x, a, b, s, *gpu_plan)
    close(y, R.lora(*(host(t) for t in (x, a, b, s)), plan, np.zeros((M, N))), lora_slack(x, a, b, s, plan, "f16"),
          "f16", "y")
    dy = normal(rng, M, N, kind="f16", size=1e-3)
    got = Z.zinc_lora_backward(dy, x, a, b, s, *gpu_plan)
    want = R.lora_backward(*(host(t) for t in (dy, x, a, b, s)), plan, np.zeros((M, K)))
    size = R.lora_backward(*(np.abs(host(t)) for t in (dy, x, a, b, s)), plan, np.zeros((M, K)))
    for g, w, z in zip(got, want, size):
        # the lower terms may be subnormal against the largest of the adapter's rows, 2^6 of their mean and less
        close(g, w, (sums(K) + sums(2 * M) + 2.0 ** -21) * z + 2.0 ** -30 * z.max(), "f16")


# ---------------------------------------------------------------- as they are used
def test_expert_layer_training_step():
    """Sort, gather, gate and up, SwiGLU, down, combine, and back: gradients against autograd in 64 bits."""
    rng = np.random.default_rng(11)
    M, k, E, H, I = 70, 2, 5, 72, 40
    x = normal(rng, M, H, kind="bf16")
    ids = rng.integers(0, E - 1, size=(M, k)).astype(np.int32)        # the last expert has no rows
    p = rng.uniform(0.2, 1, size=(M, k)).astype(np.float32)
    wg, wu = (normal(rng, E, I, H, kind="bf16", size=0.2) for _ in range(2))
    wd = normal(rng, E, H, I, kind="bf16", size=0.2)
    dy = normal(rng, M, H, kind="bf16")
    f32 = torch.float32

    offsets, slot_row, _ = Z.zinc_moe_sort(dev(ids), E)
    xs = Z.zinc_moe_gather(x, slot_row)
    g, u = (Z.zinc_moe_gemm(xs, w, offsets) for w in (wg, wu))
    h = Z.zinc_swiglu(g, u)
    ys = Z.zinc_moe_gemm(h, wd, offsets)
    y = Z.zinc_moe_combine(ys, slot_row, dev(p))
    dys, dp = Z.zinc_moe_combine_backward(dy, ys, slot_row, dev(p))
    dh, dwd = Z.zinc_moe_gemm_backward(dys, h, wd, offsets, dw_dtype=f32)
    dg, du = Z.zinc_swiglu_backward(dh, g, u)
    dxg, dwg = Z.zinc_moe_gemm_backward(dg, xs, wg, offsets, da_dtype=f32, dw_dtype=f32)
    dxu, dwu = Z.zinc_moe_gemm_backward(du, xs, wu, offsets, da_dtype=f32, dw_dtype=f32)
    dx = Z.zinc_moe_gather_backward(dxg + dxu, slot_row)

    leaves = [torch.from_numpy(host(t)).requires_grad_() for t in (x, wg, wu, wd)] + \
             [torch.from_numpy(p.astype(np.float64)).requires_grad_()]
    X, G, U, D, P = leaves
    rows = []
    for t in range(M):
        parts = []
        for s in range(k):
            e = int(ids[t, s])
            parts.append(P[t, s] * (D[e] @ (torch.nn.functional.silu(G[e] @ X[t]) * (U[e] @ X[t]))))
        rows.append(sum(parts))
    Y = torch.stack(rows)
    Y.backward(torch.from_numpy(host(dy)))
    # values are rounded to bf16 up to seven times in a row, by 2^-8 at most each: 7 2^-8 in the 2-norm
    for got, want in ((y, Y.detach()), (dx, X.grad), (dwg, G.grad), (dwu, U.grad), (dwd, D.grad), (dp, P.grad)):
        want = want.numpy()
        assert np.linalg.norm(host(got) - want) <= 7 * 2.0 ** -8 * np.linalg.norm(want)
    assert not dwg[E - 1].any() and not dwu[E - 1].any() and not dwd[E - 1].any()


def test_adapters_beside_the_fp8_projections():
    """Gate, up and down in FP8, each with adapters of one plan, SwiGLU between."""
    rng = np.random.default_rng(12)
    M, E, rank, H, I = 40, 3, 16, 256, 384
    x = activations(rng, M, H, "f16")
    ids = adapter_ids(rng, M, E)
    plan, gpu_plan = F.sort(ids.reshape(-1, 1), E), plan_of(ids, E)

    def projection(n, k):
        w = normal(rng, n, k, kind="f16", size=k ** -0.5)
        return Z.zinc_fp8_quantize(w, 128) + (normal(rng, E, rank, k, kind="f16", size=k ** -0.5),
                                              normal(rng, E, n, rank, kind="f16", size=0.3))

    def call(x, w):
        q, s, a, b = w
        y = Z.zinc_gemm_fp8(*Z.zinc_fp8_quantize(x), q, s, torch.float16)
        shared = y.clone()
        Z.zinc_lora(x, a, b, None, *gpu_plan, base=y, y=y)
        want = R.lora(host(x), host(a), host(b), np.ones(E), plan, host(shared))
        size = lora_slack(x, a, b, torch.ones(E, device=DEV), plan, "f16") + 2.0 ** -23 * np.abs(host(shared))
        close(y, want, size, "f16")
        return y

    gate, up, down = projection(I, H), projection(I, H), projection(H, I)
    h = Z.zinc_swiglu(call(x, gate), call(x, up))
    y = call(h, down)
    assert bool(y.isfinite().all())


def all_calls(s):
    """Every call of this file once, on what `s` holds."""
    out = [Z.zinc_moe_gemm(s["a"], s["w"], s["off"]), *Z.zinc_moe_gemm_backward(s["dc"], s["a"], s["w"], s["off"]),
           Z.zinc_swiglu(s["a"], s["u"]), *Z.zinc_swiglu_backward(s["dh"], s["a"], s["u"]),
           Z.zinc_lora(s["a"], s["la"], s["lb"], s["scales"], *s["plan"], base=s["base"]),
           *Z.zinc_lora_backward(s["dc"], s["a"], s["la"], s["lb"], s["scales"], *s["plan"])]
    return out


def state(seed, M, E=3, N=264, K=328, rank=24):
    rng = np.random.default_rng(seed)
    s = dict(a=activations(rng, M, K, "bf16"), u=normal(rng, M, K, kind="bf16"), dh=normal(rng, M, K, kind="bf16"),
             w=normal(rng, E, N, K, kind="bf16"), dc=normal(rng, M, N, kind="bf16"), base=normal(rng, M, N, kind="bf16"),
             off=dev(ranges(rng, M, E, outside=False)), la=normal(rng, E, rank, K, kind="bf16"),
             lb=normal(rng, E, N, rank, kind="bf16"), scales=dev(rng.uniform(size=E).astype(np.float32)),
             plan=plan_of(adapter_ids(rng, M, E), E))
    return s


@pytest.mark.parametrize("M", [3, 200, 1300])
def test_repeated_calls_give_equal_bits(M):
    s = state(M, M)
    first = all_calls(s)
    for _ in range(3):
        for a, b in zip(all_calls(s), first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [3, 1300])
def test_graph_replays(M):
    s = state(M, M)
    all_calls(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_calls(s)
    for seed in (5, 6, 7):
        new = state(seed, M)
        for name in s:
            if name == "plan":
                for t, n in zip(s[name], new[name]):
                    t.copy_(n)
            else:
                s[name].copy_(new[name])
        want = [t.clone() for t in all_calls(s)]
        torch.cuda.synchronize()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(out, want):
            assert torch.equal(got, w)


def test_side_stream_and_two_streams_at_once():
    states = [state(21, 900), state(22, 40)]
    want = [all_calls(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [[], []]
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i] = all_calls(states[i])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = states[0]
    y = Z.zinc_lora(s["a"], s["la"], s["lb"], s["scales"], *s["plan"], base=s["base"], stream=side)
    c = Z.zinc_moe_gemm(s["a"], s["w"], s["off"], stream=side)
    h = Z.zinc_swiglu(s["a"], s["u"], stream=side)
    side.synchronize()
    assert torch.equal(c, want[0][0]) and torch.equal(h, want[0][3]) and torch.equal(y, want[0][6])


def test_a_workspace_is_reused_and_its_end_kept():
    s = state(31, 700)
    M, K, N, E, rank = 700, 328, 264, 3, 24
    args = s["a"], s["la"], s["lb"], s["scales"], *s["plan"]
    need = max(Z.lora_workspace_size(M, E, K, N, rank), Z.lora_backward_workspace_size(M, E, K, N, rank))
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        assert torch.equal(Z.zinc_lora(*args, workspace=ws[:need]), Z.zinc_lora(*args))
        for a, b in zip(Z.zinc_lora_backward(s["dc"], *args, workspace=ws[:need]), Z.zinc_lora_backward(s["dc"], *args)):
            assert torch.equal(a, b)
        assert bool((ws[need:] == 0xAB).all())


# c and da in parts, da and c dealt out, dw in parts, dw dealt out, both dealt out in one launch
WITH_WORKSPACE = [(40, 1, 8, 800), (40, 2, 840, 8), (210, 300, 672, 264), (229, 130, 288, 928), (1685, 2, 8, 8),
                  (269, 300, 2616, 8), (17042, 60, 648, 688), (1088, 300, 160, 432), (3739, 20, 8, 3168)]


def product_state(seed, rows, E, N, K):
    rng = np.random.default_rng(seed)
    return (normal(rng, rows, N, kind="bf16"), normal(rng, rows, K, kind="bf16"), normal(rng, E, N, K, kind="bf16", size=0.1),
            dev(ranges(rng, rows, E, outside=False)))


def products(dc, a, w, off, forward=None, backward=None):
    return (Z.zinc_moe_gemm(a, w, off, workspace=forward),
            *Z.zinc_moe_gemm_backward(dc, a, w, off, dw_dtype=torch.float32, workspace=backward))


@pytest.mark.parametrize("rows,E,N,K", WITH_WORKSPACE)
def test_products_of_graphs_that_share_a_workspace(rows, E, N, K):
    """Two graphs on one workspace of exactly the size asked for, replayed in turn; what lies behind it is kept."""
    need = [Z.moe_gemm_workspace_size(rows, E, N, K), Z.moe_gemm_backward_workspace_size(rows, E, N, K)]
    assert max(need) > 0
    ws = torch.full((max(need) + 256,), 0xAB, dtype=torch.uint8, device=DEV)
    both = ws[:need[0]], ws[:need[1]]
    states = [product_state(seed, rows, E, N, K) for seed in (1, 2)]
    graphs, outs = [], []
    for s in states:
        products(*s)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(products(*s, *both))
    for seed in (3, 4, 5):
        want = []
        for i, s in enumerate(states):
            for t, n in zip(s, product_state(seed + 10 * i, rows, E, N, K)):
                t.copy_(n)
            want.append([t.clone() for t in products(*s)])
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for got, expected in zip(outs, want):
            for a, b in zip(got, expected):
                assert torch.equal(a, b)
        assert bool((ws[max(need):] == 0xAB).all())


@pytest.mark.parametrize("rows,E,N,K", [(17042, 60, 648, 688), (1111, 7, 520, 1032), (1685, 2, 8, 8)])
def test_gradients_of_two_types(rows, E, N, K):
    """In one launch, side by side and apart: the 16-bit gradient is the fp32 one, rounded."""
    s = product_state(7, rows, E, N, K)
    wide_a, wide_w = Z.zinc_moe_gemm_backward(*s, da_dtype=torch.float32, dw_dtype=torch.float32)
    inside = slice(int(s[3][0]), int(s[3][-1]))
    for a_type, w_type in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        da, dw = Z.zinc_moe_gemm_backward(*s, da_dtype=a_type, dw_dtype=w_type)
        assert da.dtype == a_type and dw.dtype == w_type
        assert torch.equal(da[inside], wide_a[inside].to(a_type)) and torch.equal(dw, wide_w.to(w_type))


# ---------------------------------------------------------------- past 2**32 bytes
def last_rows(rng, rows, cols, n, kind):
    """Zeros but for the last n rows."""
    x = torch.zeros((rows, cols), dtype=TYPES[kind][0], device=DEV)
    x[-n:] = normal(rng, n, cols, kind=kind)
    return x


@pytest.mark.parametrize("N,K", [(8, 640), (640, 8)])
def test_products_past_32_bits(N, K):
    rng = np.random.default_rng(N)
    rows, n = 3_600_000, 300
    a, dc, w = last_rows(rng, rows, K, n, "bf16"), last_rows(rng, rows, N, n, "bf16"), normal(rng, 2, N, K, kind="bf16")
    assert max(a.numel(), dc.numel()) * 2 > 1 << 32
    off = np.array([0, rows - 200, rows], np.int32)
    c = Z.zinc_moe_gemm(a, w, dev(off))
    da, dw = Z.zinc_moe_gemm_backward(dc, a, w, dev(off), dw_dtype=torch.float32)
    tail = np.array([0, n - 200, n], np.int32)
    at, dt, wh = host(a[-n:]), host(dc[-n:]), host(w)
    zero = lambda cols: np.zeros((n, cols))
    close(c[-n:], R.moe_gemm(at, wh, tail, zero(N)), sums(K) * R.moe_gemm(abs(at), abs(wh), tail, zero(N)), "bf16", "c")
    want = R.moe_gemm_backward(dt, at, wh, tail, zero(K))
    size = R.moe_gemm_backward(abs(dt), abs(at), abs(wh), tail, zero(K))
    close(da[-n:], want[0], sums(N) * size[0], "bf16", "da")
    close(dw, want[1], sums(n) * size[1], "f32", "dw")   # the zeros add nothing
    assert not bool(c[:-n].any()) and not bool(da[:-n].any())


def test_weights_past_32_bits():
    """The last expert's rows alone; the others' gradients are zeros."""
    rng = np.random.default_rng(3)
    E, N, K, n = 1024, 1040, 2048, 40
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
    w[-1] = normal(rng, N, K, kind="bf16")
    assert w.numel() * 2 > 1 << 32
    a, dc = normal(rng, n, K, kind="bf16"), normal(rng, n, N, kind="bf16")
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[-1] = n
    c = Z.zinc_moe_gemm(a, w, off)
    dw = torch.full_like(w, -3.0)
    da, _ = Z.zinc_moe_gemm_backward(dc, a, w, off, dw=dw)
    one, ah, dh, wh = np.array([0, n], np.int32), host(a), host(dc), host(w[-1:])
    close(c, R.moe_gemm(ah, wh, one, np.zeros((n, N))), sums(K) * R.moe_gemm(abs(ah), abs(wh), one, np.zeros((n, N))),
          "bf16", "c")
    want = R.moe_gemm_backward(dh, ah, wh, one, np.zeros((n, K)))
    size = R.moe_gemm_backward(abs(dh), abs(ah), abs(wh), one, np.zeros((n, K)))
    close(da, want[0], sums(N) * size[0], "bf16", "da")
    close(dw[-1:], want[1], sums(n) * size[1], "bf16", "dw")
    assert not bool(dw[:-1].any())


def test_rows_past_32_bits():
    """SwiGLU and the adapters: the last rows as alone."""
    rng = np.random.default_rng(5)
    rows, cols, n, rank, K = 300_000, 8192, 40, 16, 64
    gate, up, base = (last_rows(rng, rows, cols, n, "bf16") for _ in range(3))
    assert gate.numel() * 2 > 1 << 32
    assert torch.equal(Z.zinc_swiglu(gate, up)[-n:], Z.zinc_swiglu(gate[-n:], up[-n:]))
    for got, want in zip(Z.zinc_swiglu_backward(base, gate, up), Z.zinc_swiglu_backward(base[-n:], gate[-n:], up[-n:])):
        assert torch.equal(got[-n:], want)
    x = last_rows(rng, rows, K, n, "bf16")
    a, b = normal(rng, 2, rank, K, kind="bf16"), normal(rng, 2, cols, rank, kind="bf16", size=0.1)
    ids = np.full(rows, -1)
    ids[-n:] = rng.integers(-1, 2, n)
    y = Z.zinc_lora(x, a, b, None, *plan_of(ids, 2), base=base)
    want = Z.zinc_lora(x[-n:].contiguous(), a, b, None, *plan_of(ids[-n:], 2), base=base[-n:].contiguous())
    assert torch.equal(y[-n:], want) and not bool(y[:-n].any())
    # gradients, with the wide matrix as x
    wide, tall = b.transpose(1, 2).contiguous(), a.transpose(1, 2).contiguous()
    back = Z.zinc_lora_backward(x, base, wide, tall, None, *plan_of(ids, 2))
    tail = F.sort(ids[-n:].reshape(-1, 1).astype(np.int32), 2)
    args = [host(t) for t in (x[-n:], base[-n:], wide, tall)] + [np.ones(2)]
    want = R.lora_backward(*args, tail, np.zeros((n, cols)))
    size = R.lora_backward(*(np.abs(t) for t in args), tail, np.zeros((n, cols)))
    each = split_off("bf16") + 4 * 2.0 ** -24
    assert not bool(back[0][:-n].any())
    close(back[0][-n:], want[0], (sums(K) + sums(2 * rank) + each) * size[0], "bf16", "dx")
    close(back[1], want[1], (sums(K) + sums(2 * n + 64) + each) * size[1], "bf16", "da")
    close(back[2], want[2], (sums(cols) + sums(2 * n + 64) + each) * size[2], "bf16", "db")
