"""The float64 definitions of the products by expert, SwiGLU and the adapters against loops and differences."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.fp8 as F
import oracle.rows16 as R


def differences(f, x, d=1e-5):
    """The gradient of the number f(x) by central differences."""
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + d
        up = f(x)
        x[i] = keep - d
        g[i] = (up - f(x)) / (2 * d)
        x[i] = keep
    return g


def test_products_by_loops():
    rng = np.random.default_rng(1)
    a, w = rng.standard_normal((7, 4)), rng.standard_normal((3, 5, 4))
    offsets = [1, 4, 4, 6]
    c = R.moe_gemm(a, w, offsets, np.full((7, 5), 9.0))
    expert = [None, 0, 0, 0, 2, 2, None]
    for r, e in enumerate(expert):
        for n in range(5):
            want = 9.0 if e is None else sum(a[r, k] * w[e, n, k] for k in range(4))
            assert c[r, n] == pytest.approx(want, abs=1e-12)


def test_offsets_are_cut():
    rng = np.random.default_rng(2)
    a, w = rng.standard_normal((4, 3)), rng.standard_normal((2, 2, 3))
    c = R.moe_gemm(a, w, [-5, 2, 99], np.zeros((4, 2)))
    assert np.allclose(c, np.concatenate([a[:2] @ w[0].T, a[2:] @ w[1].T]))


def test_product_gradients_by_differences():
    rng = np.random.default_rng(3)
    a, w, dc = rng.standard_normal((6, 3)), rng.standard_normal((3, 4, 3)), rng.standard_normal((6, 4))
    offsets = [0, 2, 2, 5]
    da, dw = R.moe_gemm_backward(dc, a, w, offsets, np.zeros((6, 3)))
    inside = np.arange(6) < 5
    value = lambda a, w: float((R.moe_gemm(a, w, offsets, np.zeros((6, 4))) * dc)[inside].sum())  # noqa: E731
    assert np.allclose(da, differences(lambda v: value(v, w), a), atol=1e-8)
    assert np.allclose(dw, differences(lambda v: value(a, v), w), atol=1e-8)
    assert not dw[1].any()


def test_swiglu_and_its_gradients():
    rng = np.random.default_rng(4)
    g, u, dh = (3 * rng.standard_normal((3, 5)) for _ in range(3))
    assert np.allclose(R.swiglu(g, u), g / (1 + np.exp(-g)) * u)
    dg, du = R.swiglu_backward(dh, g, u)
    assert np.allclose(dg, differences(lambda v: float((R.swiglu(v, u) * dh).sum()), g), atol=1e-7)
    assert np.allclose(du, differences(lambda v: float((R.swiglu(g, v) * dh).sum()), u), atol=1e-7)


def test_adapters_by_rows_and_differences():
    rng = np.random.default_rng(5)
    M, E, r, K, N = 6, 3, 2, 4, 5
    x, base, dy = rng.standard_normal((M, K)), rng.standard_normal((M, N)), rng.standard_normal((M, N))
    a, b, scales = rng.standard_normal((E, r, K)), rng.standard_normal((E, N, r)), rng.uniform(0.5, 2, E)
    ids = np.array([[2], [0], [-1], [2], [0], [7]], dtype=np.int32)
    plan = F.sort(ids, E)
    y = R.lora(x, a, b, scales, plan, base)
    for m, e in enumerate(ids[:, 0]):
        want = base[m] + (scales[e] * b[e] @ (a[e] @ x[m]) if 0 <= e < E else 0)
        assert np.allclose(y[m], want)
    dx, da, db = R.lora_backward(dy, x, a, b, scales, plan, np.zeros((M, K)))
    value = lambda x, a, b: float((R.lora(x, a, b, scales, plan, base) * dy).sum())  # noqa: E731
    assert np.allclose(dx, differences(lambda v: value(v, a, b), x), atol=1e-7)
    assert np.allclose(da, differences(lambda v: value(x, v, b), a), atol=1e-7)
    assert np.allclose(db, differences(lambda v: value(x, a, v), b), atol=1e-7)
    assert not da[1].any() and not db[1].any()
