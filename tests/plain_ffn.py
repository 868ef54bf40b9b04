"""Plain 64-bit definitions (numpy) of the experts' feed-forward products and
their gradients, the combine's gradients and the projection with adapters,
each with a bound of the rounding errors that the GPU's arithmetic may make.

The bounds, from the arithmetic:

* products of two bfloat16 are exact in binary32; each of the k additions may
  be off by 2^-23 of the sum of magnitudes (the matrix unit's own order);
* exp(-g) in binary32: the argument's rounding (|g| 1.45 2^-24) and the
  result's, with the reciprocal and the products after it: relative
  (16 + 2 |g|) 2^-24 on sigmoid(g);
* the outputs' rounding: half a step, 2^-8 of the value in bfloat16 and 2^-24 in
  binary32, and what lies below the smallest normal numbers (2^-126) may go.
"""
from __future__ import annotations

import numpy as np

ADD, TINY = 2.0**-23, 2.0**-125
STEP = {"bf16": 2.0**-8, "f32": 2.0**-24}


def rounded(v, err, out):
    """Bound on an output of value v that was off by err before its rounding."""
    return err + STEP[out] * (np.abs(v) + err) + TINY


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + e), e / (1 + e))


def sigmoid_error(g):
    return (16 + 2 * np.abs(g)) * 2.0**-24


def product(a, w):
    """(a w^T, error)."""
    return a @ w.T, len(w.T) * ADD * (np.abs(a) @ np.abs(w).T)


def gated(a, w):
    """w = [gate rows; up rows]: (g, eg, u, eu, h, eh)."""
    n = len(w) // 2
    g, eg = product(a, w[:n])
    u, eu = product(a, w[n:])
    s = sigmoid(g)
    h = g * s * u
    # |silu'| <= 1.1
    eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(g * s) * eu + np.abs(h) * (sigmoid_error(g) + 2.0**-22)
    return g, eg, u, eu, h, eh


def row_grad(dy, w):
    """(dy w, error)."""
    return dy @ w, len(w) * ADD * (np.abs(dy) @ np.abs(w))


def gate_grad(dy, w, g, u):
    """Gradients of the rows [g | u] of silu(g) u: (dg, e, du, e)."""
    d, ed = row_grad(dy, w)
    s = sigmoid(g)
    slope = s * (1 + g * (1 - s))
    rel = sigmoid_error(g) + 2.0**-21
    dg, du = d * u * slope, d * g * s
    # 1 + g (1 - s) may cancel: its error is that of its terms
    e_dg = ed * np.abs(u * slope) + np.abs(d * u * s) * (1 + np.abs(g) * (1 - s)) * rel * 2
    e_du = ed * np.abs(g * s) + np.abs(du) * rel
    # 1 - s is a difference of two values below 1
    e_dg += np.abs(d * u * s * g) * 2.0**-22
    return dg, e_dg, du, e_du


def weight_grad(dy, a):
    """(dy^T a, error)."""
    return dy.T @ a, max(len(dy), 1) * ADD * (np.abs(dy).T @ np.abs(a))


def combine(pos, w, y_exp):
    return (w[:, :, None] * y_exp[pos]).sum(axis=1)


def combine_grad(pos, w, dy, y_exp):
    """(dy_exp rows by pair [N, K, H], dw, error of dw)."""
    rows = w[:, :, None] * dy[:, None, :]
    dw = np.einsum("nh,nkh->nk", dy, y_exp[pos])
    mag = np.einsum("nh,nkh->nk", np.abs(dy), np.abs(y_exp[pos]))
    return rows, dw, dy.shape[1] * ADD * mag


def lora(x, w, a, b, scale, adapter):
    """(y, error): a projection with one adapter or none for each row."""
    y, ey = product(x, w)
    L, r, k = a.shape
    for t, i in enumerate(adapter):
        if 0 <= i < L:
            v = scale[i] * (a[i] @ x[t])
            ev = np.abs(scale[i]) * (k + 8) * ADD * (np.abs(a[i]) @ np.abs(x[t]))
            y[t] += b[i] @ v
            ey[t] += np.abs(b[i]) @ (ev + (4 * r + 8) * ADD * np.abs(v))
    return y, ey
