"""The float64 definitions of the FP8 expert layer (oracle/fp8.py) against things
other than themselves: torch's e4m3 type, closed forms, brute force and
differences.  CPU only."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
import oracle.fp8 as F


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = F.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_e4m3_encode_rounds_to_nearest_even_as_torch_does():
    v = F.e4m3_values()
    pos = v[:127]
    mid = (pos[1:] + pos[:-1]) / 2                                   # every tie
    near = np.concatenate([pos, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), np.linspace(0, 448, 5003)])
    near = near.astype(np.float32)
    both = np.concatenate([near, -near])
    want = torch.from_numpy(both).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(F.e4m3_encode(both), want)
    assert np.array_equal(F.e4m3_encode(np.array([np.nan, np.inf])), [0x7F, 0x7F])


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.0001, 2.0), (449.0, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
                                        (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (0.0, 1.0), (1e30, 2.0 ** 91),
                                        (2.0 ** -140, 2.0 ** -126)])
def test_scales_in_closed_form(amax, scale):
    x = np.zeros((1, 130))
    x[0, 7] = -amax
    x[0, 129] = 448.0 * 8
    assert F.block_scales(x, 1).tolist() == [[scale, 8.0]]
    assert F.block_scales(np.repeat(x, 130, axis=0), 128).shape == (2, 2)


def test_quantize_is_exact_on_its_own_values_and_within_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((9, 272)) * np.exp(rng.standard_normal((9, 1)))
    q, s = F.quantize(x)
    back = F.dequantize(q, s, 1)
    step = np.maximum(np.abs(back), F.spread(s, 1, x.shape) * 2.0 ** -6) * 2.0 ** -3
    assert np.all(np.abs(back - x) <= step / 2 * (1 + 1e-12))
    q2, _ = F.quantize(back)
    assert np.array_equal(F.dequantize(q2, _, 1), back)              # idempotent in value
    assert np.array_equal(F.quantize(x * 4)[0], q) and np.array_equal(F.quantize(x * 4)[1], 4 * s)


def test_sort_brute_force_and_invalid_ids():
    rng = np.random.default_rng(4)
    ids = rng.integers(-2, 9, size=(23, 3)).astype(np.int32)
    off, slot_row, row_slot = F.sort(ids, 7)
    flat = ids.reshape(-1)
    valid = [i for i in range(flat.size) if 0 <= flat[i] < 7]
    assert row_slot[:len(valid)].tolist() == sorted(valid, key=lambda i: (flat[i], i))
    assert np.all(row_slot[len(valid):] == -1) and off[-1] == len(valid)
    assert all(off[e + 1] - off[e] == np.sum(flat == e) for e in range(7))
    for i, r in enumerate(slot_row.reshape(-1)):
        assert (r == -1) if i not in valid else row_slot[r] == i


def test_combine_inverts_gather_and_gradients_are_differences():
    rng = np.random.default_rng(5)
    M, k, H, E = 6, 3, 8, 4
    ids = rng.integers(-1, E, size=(M, k))
    _, slot_row, _ = F.sort(ids, E)
    x = rng.standard_normal((M, H))
    xs = F.gather(x, slot_row, np.full((M * k, H), 7.0))
    uses = (slot_row >= 0).sum(1, keepdims=True)
    assert np.allclose(F.combine(xs, slot_row, None), uses * x, rtol=1e-14)
    # <combine(ys), dy> against differences in ys and in the weights
    ys, p, dy = rng.standard_normal((M * k, H)), rng.uniform(size=(M, k)), rng.standard_normal((M, H))
    dys, dp = F.combine_backward(dy, ys, slot_row, p, np.zeros((M * k, H)))
    f = lambda a, b: float((F.combine(a, slot_row, b) * dy).sum())
    eps = 1e-6
    for _ in range(20):
        i, j = rng.integers(M * k), rng.integers(H)
        d = np.zeros_like(ys)
        d[i, j] = eps
        assert abs((f(ys + d, p) - f(ys - d, p)) / (2 * eps) - dys[i, j]) < 1e-8
        t, s = rng.integers(M), rng.integers(k)
        d = np.zeros_like(p)
        d[t, s] = eps
        assert abs((f(ys, p + d) - f(ys, p - d)) / (2 * eps) - dp[t, s]) < 1e-8
    # the gather's gradient is the plain sum: <gather(x), dxs> is linear in x
    dxs = rng.standard_normal((M * k, H))
    named = slot_row[slot_row >= 0]
    dx = F.combine(dxs, slot_row, None)
    assert np.isclose((x * dx).sum(), (xs[named] * dxs[named]).sum(), rtol=1e-12)


def test_gemm_brute_force_with_cut_blocks():
    rng = np.random.default_rng(6)
    M, N, K = 3, 130, 144
    a, w = (rng.integers(0, 0x7F, size=(r, K)).astype(np.uint8) for r in (M, N))
    sa, sw = rng.uniform(0.5, 2, size=(M, 2)), rng.uniform(0.5, 2, size=(2, 2))
    c = F.gemm(a, sa, w, sw)
    va, vw = F.e4m3_decode(a), F.e4m3_decode(w)
    for m, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        want = sum(va[m, k] * sa[m, k // 128] * vw[n, k] * sw[n // 128, k // 128] for k in range(K))
        assert np.isclose(c[m, n], want, rtol=1e-12)


def test_experts_reduce_to_one_dense_mlp():
    rng = np.random.default_rng(7)
    H, I, M = 128, 256, 5
    gate, up, down = (F.quantize(rng.standard_normal(s), 128) for s in ((I, H), (I, H), (H, I)))
    x = rng.standard_normal((M, H)).astype(np.float16)
    stack = lambda q: (q[0][None], q[1][None])
    y, slots = F.experts(stack(gate), stack(up), stack(down), x, np.zeros((M, 1), np.int32), np.ones((M, 1)))
    xq = F.dequantize(*F.quantize(x), 1)
    h = O.silu(xq @ F.dequantize(*gate, 128).T) * (xq @ F.dequantize(*up, 128).T)
    assert np.allclose(y, F.dequantize(*F.quantize(h), 1) @ F.dequantize(*down, 128).T, rtol=1e-12)
    assert len(slots) == M
    none, slots = F.experts(stack(gate), stack(up), stack(down), x, np.full((M, 1), 1), np.ones((M, 1)))
    assert not none.any() and not slots
