"""Plain float64 definitions of the products by expert, SwiGLU and the low-rank adapters, with their
gradients (numpy), written from the formulas.  No code is shared with the HIP path.

``offsets`` holds the first row of each expert and, last, the end; ``plan`` is the sort's
``(offsets, slot_row, row_slot)`` of the rows' adapter ids.
"""
from __future__ import annotations

import numpy as np


def _ranges(offsets, rows):
    at = np.clip(np.asarray(offsets, dtype=np.int64), 0, rows)
    return [slice(at[e], max(at[e], at[e + 1])) for e in range(len(at) - 1)]


def moe_gemm(a, w, offsets, c):
    """c with the rows inside the ranges replaced by a's times their expert's w."""
    c = np.array(c, dtype=np.float64)
    for e, at in enumerate(_ranges(offsets, len(a))):
        c[at] = a[at] @ w[e].T
    return c


def moe_gemm_backward(dc, a, w, offsets, da):
    da, dw = np.array(da, dtype=np.float64), np.zeros(w.shape)
    for e, at in enumerate(_ranges(offsets, len(a))):
        da[at] = dc[at] @ w[e]
        dw[e] = dc[at].T @ a[at]
    return da, dw


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def swiglu(gate, up):
    return gate * sigmoid(gate) * up


def swiglu_backward(dh, gate, up):
    s = sigmoid(gate)
    return dh * up * s * (1.0 + gate * sigmoid(-gate)), dh * gate * s


def lora(x, a, b, scales, plan, base):
    """base plus, for each row in the plan, its adapter's product."""
    offsets, _, row_slot = plan
    y = np.array(base, dtype=np.float64)
    for e, at in enumerate(_ranges(offsets, len(x))):
        rows = row_slot[at]
        y[rows] += scales[e] * ((x[rows] @ a[e].T) @ b[e].T)
    return y


def lora_backward(dy, x, a, b, scales, plan, base):
    offsets, _, row_slot = plan
    dx, da, db = np.array(base, dtype=np.float64), np.zeros(a.shape), np.zeros(b.shape)
    for e, at in enumerate(_ranges(offsets, len(x))):
        rows = row_slot[at]
        dh = scales[e] * (dy[rows] @ b[e])
        dx[rows] += dh @ a[e]
        da[e] = dh.T @ x[rows]
        db[e] = scales[e] * (dy[rows].T @ (x[rows] @ a[e].T))
    return dx, da, db
