"""Plain 64-bit definitions of the router, the norm, the 4-bit rows and the
experts' products (numpy), for the tests of the GPU kernels."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_round(a: np.ndarray) -> np.ndarray:
    """float32 values rounded to the nearest bfloat16 (ties to even), as float32."""
    b = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    out = r.view(np.float32).copy()
    out[np.isnan(a)] = np.nan
    return out


def route(logits, k, score="softmax", bias=None, n_groups=1, top_groups=1, group_top=1, renorm=True,
          scale=1.0):
    """(ids, w) of every row: one token at a time, from the definition."""
    l = np.asarray(logits, np.float64)
    n, e = l.shape
    ids, w = np.zeros((n, k), np.int32), np.zeros((n, k))
    b = np.zeros(e) if bias is None else np.asarray(bias, np.float64)
    size = e // n_groups
    for t in range(n):
        x = l[t].copy()
        off = np.isnan(x) | (x == -np.inf)  # masked by the logit
        mask = off | np.isnan(b) | (b == -np.inf)
        s = np.zeros(e)
        live = ~off
        if score == "softmax":
            if live.any():
                m = x[live].max()
                d = np.where(x[live] == m, 0.0, x[live] - m)
                s[live] = np.exp(d) / np.exp(d).sum()
        else:
            p = x[live]
            ex = np.exp(-np.abs(p))
            s[live] = np.where(p >= 0, 1 / (1 + ex), ex / (1 + ex))
        # scores rise with the logits: without a bias (and with maxima for
        # group scores) the order is that of the logits themselves
        by_logit = bias is None and (top_groups == n_groups or group_top == 1)
        choice = np.where(mask, -np.inf, x if by_logit else s + np.where(mask, 0, b))
        closed = np.zeros(e, bool)
        if top_groups < n_groups:
            by = np.sort(choice.reshape(n_groups, size), axis=1)[:, ::-1]
            gs = np.where(by[:, group_top - 1] > -np.inf, by[:, :group_top].sum(axis=1), -np.inf)
            keep = sorted(range(n_groups), key=lambda g: (-gs[g], g))[:top_groups]
            closed = ~np.isin(np.arange(e) // size, keep)
        order = sorted((i for i in range(e) if not closed[i]), key=lambda i: (-choice[i], i))[:k]
        ids[t] = order
        live_k = ~mask[order]
        if not live_k.any():
            continue
        if renorm:  # shifted by the largest chosen logit, so that nothing underflows
            p = x[order][live_k]
            if score == "softmax":
                v = np.exp(np.where(p == p.max(), 0.0, p - p.max()))
            else:
                lo = np.minimum(p, 0.0)
                v = np.exp(lo - lo.max()) / (1 + np.exp(-np.abs(p)))
            w[t, live_k] = v / v.sum() * scale
        else:
            w[t, live_k] = s[order][live_k] * scale
    return ids, w


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    """OCP fp8 e4m3fn codes as float64."""
    c = np.arange(256)
    man, ex = c & 7, (c >> 3) & 15
    v = np.where(ex == 0, man / 8 * 2.0**-6, (1 + man / 8) * 2.0 ** (ex - 7))
    v = np.where((c & 127) == 127, np.nan, v) * np.where(c & 128, -1.0, 1.0)
    return v[codes]


def rmsnorm(x, weight, eps, residual=None):
    """(h, y, scale): the sum, the normed rows and their scale per 128."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    ms = (h * h).mean(axis=1, keepdims=True) + eps
    y = h / np.sqrt(np.where(ms > 0, ms, 1.0)) * np.asarray(weight, np.float64)
    amax = np.abs(y.reshape(len(y), -1, 128)).max(axis=2)
    return h, y, np.where(amax < 2.0**-110, 1.0, amax / 448)


def mx4_scale_bytes(v: np.ndarray) -> np.ndarray:
    """Scale byte of every block of 32 of float64 rows [m, h]."""
    b = np.abs(v.reshape(len(v), -1, 32))
    bad = ~np.isfinite(b).all(axis=2)
    amax = np.where(bad, 1.0, np.where(np.isfinite(b), b, 0).max(axis=2))
    ex = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1
    s = np.clip(127 + ex - 2, 0, 254)
    return np.where(bad, 255, np.where(amax > 0, s, 0)).astype(np.uint8)


def mx4_codes(v: np.ndarray, s: np.ndarray) -> np.ndarray:
    """Element codes [m, h] (sign in bit 3) of float64 rows under scale bytes:
    the nearest of the eight magnitudes, ties to the even code."""
    m, h = v.shape
    u = v.reshape(m, -1, 32) / 2.0 ** (s.astype(np.float64) - 127)[:, :, None]
    u = np.where((s == 255)[:, :, None], 0.0, u)
    a = np.abs(u)
    d = np.abs(a[..., None] - E2M1)
    low = d.argmin(axis=-1)  # the lower of two equally near
    up = np.minimum(low + 1, 7)
    tie = np.take_along_axis(d, low[..., None], -1)[..., 0] == np.take_along_axis(
        d, up[..., None], -1)[..., 0]
    code = np.where(tie & (low % 2 == 1) & (up != low), up, low)
    sign = np.signbit(u) & (s != 255)[:, :, None]
    return (code + 8 * sign).reshape(m, h).astype(np.uint8)


def pack4(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def mx4_values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    """float64 rows of packed codes [m, h/2] and scale bytes [m, h/32]."""
    codes = np.stack((q & 15, q >> 4), axis=-1).reshape(len(q), -1)
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    unit = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return v * np.repeat(unit, 32, axis=1)


def swiglu(x: np.ndarray) -> np.ndarray:
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    return g / (1 + np.exp(-g)) * u


def slots(cu, rep, P, Eh, R, cap):
    """(expert, first row, past the last) of every slot that holds rows."""
    out = []
    for r in range(P):
        for i in range(Eh + R):
            lo, hi = int(cu[r][i]), int(cu[r][i + 1])
            e = r * Eh + i if i < Eh else int(rep[r][i - Eh])
            if hi > lo and e >= 0:
                out.append((e, r * cap + lo, r * cap + hi))
    return out


def expert(a, w, groups, n):
    """(y, mag, used): rows of every slot times its expert's weights
    (a [rows, k], w [E, n, k], float64), sum |a w| and the rows written."""
    y, mag = np.zeros((len(a), n)), np.zeros((len(a), n))
    used = np.zeros(len(a), bool)
    for e, lo, hi in groups:
        y[lo:hi] = a[lo:hi] @ w[e].T
        mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w[e]).T
        used[lo:hi] = True
    return y, mag, used
