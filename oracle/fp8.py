"""Plain float64 definitions of the FP8 expert layer (numpy), written from the
formulas: e4m3 values, the block quantiser, the sort of routed slots, the
weighted way back and its gradients, block-scaled products and the expert MLP.
No code is shared with the HIP path.

e4m3: sign, four exponent bits (bias 7), three fraction bits; exponent field 0 is
subnormal (steps of 2^-9), field 15 reaches 448 (fraction 6), and fraction 7 of
it is NaN; there are no infinities.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3_values() -> np.ndarray:
    """The 256 values of the e4m3 codes (NaN at 0x7F and 0xFF)."""
    code = np.arange(256)
    field, frac = (code >> 3) & 15, code & 7
    mag = np.where(field == 0, frac * 2.0 ** -9, (8 + frac) * 2.0 ** (field - 10.0))
    mag = np.where((code & 0x7F) == 0x7F, np.nan, mag)
    return np.where(code & 0x80, -mag, mag)


_VALUES = e4m3_values()


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    return _VALUES[np.asarray(codes, dtype=np.uint8)]


def e4m3_encode(v: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values, ties to the even code; |v| <= 448, or not finite (NaN code)."""
    v = np.asarray(v, dtype=np.float64)
    pos = _VALUES[:127]                                # ascending, 0 .. 448
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    hi = np.minimum(np.searchsorted(pos, a), 126)      # first value >= a
    lo = np.maximum(hi - 1, 0)
    dh, dl = pos[hi] - a, a - pos[lo]
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isfinite(v), code, 0x7F)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def _blocks(x: np.ndarray, block_rows: int) -> np.ndarray:
    R, C = x.shape
    rb, cb = -(-R // block_rows), -(-C // 128)
    p = np.zeros((rb * block_rows, cb * 128))
    p[:R, :C] = x
    return p.reshape(rb, block_rows, cb, 128)


def block_scales(x: np.ndarray, block_rows: int) -> np.ndarray:
    """The smallest powers of two s (at least 2^-126) with max|x| <= 448 s over the finite values of each
    block_rows x 128 block; 1 where all of them are zero."""
    p = _blocks(np.asarray(x, dtype=np.float64), block_rows)
    amax = np.abs(np.where(np.isfinite(p), p, 0.0)).max(axis=(1, 3))
    s = np.full(amax.shape, 2.0 ** -126)
    while np.any(need := amax > E4M3_MAX * s):
        s = np.where(need, 2.0 * s, s)
    return np.where(amax > 0, s, 1.0)


def spread(scales: np.ndarray, block_rows: int, shape) -> np.ndarray:
    """One scale per element of a [..., rows, cols] matrix."""
    s = np.asarray(scales, dtype=np.float64)
    return np.repeat(np.repeat(s, block_rows, axis=-2), 128, axis=-1)[..., :shape[-2], :shape[-1]]


def quantize(x: np.ndarray, block_rows: int = 1):
    """(codes uint8, scales) of x."""
    x = np.asarray(x, dtype=np.float64)
    s = block_scales(x, block_rows)
    return e4m3_encode(x / spread(s, block_rows, x.shape)), s


def dequantize(codes: np.ndarray, scales: np.ndarray, block_rows: int) -> np.ndarray:
    return e4m3_decode(codes) * spread(scales, block_rows, np.shape(codes))


def sort(ids: np.ndarray, n_experts: int):
    """(offsets, slot_row, row_slot) as zinc_moe_sort defines them."""
    flat = np.asarray(ids).reshape(-1)
    slot_row = np.full(flat.shape, -1, dtype=np.int32)
    row_slot = np.full(flat.shape, -1, dtype=np.int32)
    offsets = np.zeros(n_experts + 1, dtype=np.int32)
    row = 0
    for e in range(n_experts):
        for i in np.nonzero(flat == e)[0]:
            slot_row[i], row_slot[row] = row, i
            row += 1
        offsets[e + 1] = row
    return offsets, slot_row.reshape(np.shape(ids)), row_slot


def gather(x: np.ndarray, slot_row: np.ndarray, out: np.ndarray) -> np.ndarray:
    for t, rows in enumerate(slot_row):
        for r in rows:
            if r >= 0:
                out[r] = x[t]
    return out


def combine(ys: np.ndarray, slot_row: np.ndarray, weights: np.ndarray | None) -> np.ndarray:
    ys = np.asarray(ys, dtype=np.float64)
    y = np.zeros((slot_row.shape[0], ys.shape[1]))
    for t, rows in enumerate(slot_row):
        for s, r in enumerate(rows):
            if r >= 0:
                y[t] += ys[r] * (1.0 if weights is None else float(weights[t, s]))
    return y


def combine_backward(dy: np.ndarray, ys: np.ndarray, slot_row: np.ndarray, weights: np.ndarray, dys: np.ndarray):
    """(dys with the named rows written, dweights)."""
    dy, ys = np.asarray(dy, dtype=np.float64), np.asarray(ys, dtype=np.float64)
    dp = np.zeros(slot_row.shape)
    for t, rows in enumerate(slot_row):
        for s, r in enumerate(rows):
            if r >= 0:
                dys[r] = float(weights[t, s]) * dy[t]
                dp[t, s] = dy[t] @ ys[r]
    return dys, dp


def gemm(a, a_scales, w, w_scales) -> np.ndarray:
    """a codes [M, K] times w codes [N, K] transposed, each with its scales."""
    return dequantize(a, a_scales, 1) @ dequantize(w, w_scales, 128).T


def silu(z: np.ndarray) -> np.ndarray:
    return z / (1.0 + np.exp(-z))


def experts(gate, up, down, x, ids, weights):
    """The FP8 expert layer; gate, up, down: (codes [E, rows, cols], scales).  Returns y float64 and, for each
    slot of a valid expert, its (token, weight, expert, h before its quantisation)."""
    x = np.asarray(x, dtype=np.float64)
    xq = dequantize(*quantize(x), 1)
    E = gate[0].shape[0]
    y, slots = np.zeros(x.shape), []
    for t in range(x.shape[0]):
        for s in range(ids.shape[1]):
            e = int(ids[t, s])
            if 0 <= e < E:
                slots.append((t, float(weights[t, s]), e))
    hs = [None] * len(slots)
    for e in range(E):
        mine = [i for i, v in enumerate(slots) if v[2] == e]
        if not mine:
            continue
        rows = xq[[slots[i][0] for i in mine]]
        g = rows @ dequantize(gate[0][e], gate[1][e], 128).T
        u = rows @ dequantize(up[0][e], up[1][e], 128).T
        h = silu(g) * u
        out = dequantize(*quantize(h), 1) @ dequantize(down[0][e], down[1][e], 128).T
        for j, i in enumerate(mine):
            t, p, _ = slots[i]
            y[t] += p * out[j]
            hs[i] = h[j]
    return y, [(t, p, e, h) for (t, p, e), h in zip(slots, hs)]
