"""Corners of the experts' products from bf16 rows, their gradients, the
combine's gradients and the projection with adapters on the GPU: infinities
value by value, plans that do not fit their sizes, far gates, offsets past
2^31 elements, launches that go round, and many slots."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import token_dispatch_mb_amd as mb

from . import gpu_harness as G
from . import plain_ffn as F
from . import plain_ops as R
from .test_gpu_ffn import MARK, Layer, bf, dev, f64, marked, near, out, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_required():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def ints(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(G.dev())


# ------------------------------------------------------------ adapters

@pytest.mark.parametrize("order", ["turns", "runs"])
@pytest.mark.parametrize("t,n,k", [
    (4, 72, 72), (16, 520, 520),  # operands straight from memory
    (64, 1032, 1032),             # tiles in parts
    (300, 520, 136), (4400, 4360, 72),  # tiles of 128 and 256 rows, the reduction in one
])
def test_lora_infinities_keep_their_sign(t, n, k, order):
    """What an infinite element of an adapter gives is what the formula does,
    however few bits its factor has: an infinity, NaN where the factor is zero
    or infinities of both signs meet; and the same in every kernel."""
    r = rng(t, n, 11)
    ad = np.arange(t) % 4 - 1 if order == "turns" else np.arange(t) * 4 // t - 1
    x, w = bf(r, t, k), bf(r, n, k)
    # factors of one to 24 bits, zeros among them: adapter 0's inner sums are
    # x's first eight elements, 1's are those times a scale of 14 bits
    x[:, :8] = np.array([1, -1, 1.5, 0, 2.0**-20, -2.0**30, 1.0078125, -0.75])[
        r.integers(0, 8, (t, 8))]
    a, b = np.zeros((3, 8, k)), bf(r, 3, n, 8)
    a[0, np.arange(8), np.arange(8)] = a[1, np.arange(8), np.arange(8)] = 1
    scale = np.array([1.0, 1 + 2.0**-13, 0.5])
    for i in (0, 1):
        for sign in (np.inf, -np.inf):
            b[i, r.integers(0, n, max(n // 6, 2)), r.integers(0, 8, max(n // 6, 2))] = sign
    # adapter 2: its rows' inner sums are infinite themselves where x is
    a[2], b[2] = 1, np.abs(b[2]) + 1
    b[2, ::3, 1] = np.inf
    infinite = (ad == 2) & (np.arange(t) % 3 == 0)
    x[infinite, 5], w[:, 5] = np.inf, np.abs(w[:, 5]) + 1
    w, b = (R.bf16_round(np.float32(m)).astype(np.float64) for m in (w, b))  # as the GPU has them
    v = np.where((ad == 2)[:, None], x.sum(axis=1)[:, None], x[:, :8])
    v = np.float32(v * np.where(ad >= 0, scale[ad], 0)[:, None]).astype(np.float64)
    # only adapters 0 and 1 have exact inner sums
    fin = np.where(infinite[:, None], 0, x)
    want, err = F.product(fin, w)
    want[infinite] = np.inf
    mag = np.zeros_like(want)
    with np.errstate(invalid="ignore"):
        for q in range(8):
            part = np.where((ad >= 0)[:, None], v[:, q:q + 1] * b[ad][:, :, q], 0)
            want = want + part
            mag += np.abs(part)
        err = err * (1 + 40 / k) + mag * (40 + k) * F.ADD  # up to 24 additions more, and of the parts
    prm = mb.LoraParams.make(t, n, k, 8, 3, dtype_out="f32")
    y = out(t, n, dtype="f32")
    mb.project_lora(prm, dev(x), dev(w), dev(a), dev(b), dev(scale, torch.float32), ints(ad),
                    mb.alloc_lora_workspace(prm, G.dev()), y)
    got = f64(y)
    for kind in (np.isnan, np.isposinf, np.isneginf):
        bad = kind(got) != kind(want)
        assert not bad.any(), (kind.__name__, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                               got[bad][:4], want[bad][:4])
    good = np.isfinite(want) & (ad != 2)[:, None]
    near(got[good], want[good], F.rounded(want, err, "f32")[good])


# ------------------------------------------------------------ weights' gradients

@pytest.mark.parametrize("add", [False, True])
def test_wgrad_without_tokens_takes_no_rows_of_another_plan(add):
    L = Layer([[37, 0, 5, 1], [0, 70, 13, 2]], 3)
    d = mb.Dims.make(0, 1, L.E, L.P, L.R, 128, cap=L.cap)
    n, k = 72, 40
    ones = torch.ones(L.rows, n, dtype=torch.bfloat16, device=G.dev())
    dw = out(L.E, n, k, dtype="f32")
    mb.expert_bf16_wgrad(d, L.bufs, n, k, ones, ones, dw, accumulate=add)
    assert marked(dw).all() if add else not f64(dw).any()


# ------------------------------------------------------------ far gates

@pytest.mark.parametrize("rows", [3, 64, 300])
def test_far_gates_of_large_ups_keep_their_value(rows):
    """silu(g) u where silu(g) alone is below binary32 and u brings it back."""
    gates = np.array([-170, -150, -130, -110, -104, -95, -88.5, -81, -60, -3, 0.5, 90])
    ups = 2.0 ** np.array([0, 30, 60, 90, 120])
    n, k = len(gates) * len(ups) + 4, 8
    pair = np.array([(g, u) for g in gates for u in ups] + [(1, 1)] * 4)
    pair = R.bf16_round(np.float32(pair)).astype(np.float64)
    L = Layer([[rows]], 1)
    a = np.zeros((rows, k))
    a[:, 0] = 1
    w = np.zeros((1, 2 * n, k))
    w[0, :n, 0], w[0, n:, 0] = pair.T
    y = out(rows, n)
    mb.expert_bf16(L.dims, L.bufs, n, k, dev(a), dev(w), y, act="swiglu")
    g, u = pair.T
    h = g * F.sigmoid(g) * u
    # the products of the sums are exact here; the exponential's argument and
    # result, the reciprocal, four products
    want = np.broadcast_to(h, (rows, n))
    fits = np.abs(h) < 2.0**127
    near(f64(y)[:, fits], want[:, fits],
         F.rounded(want, np.abs(want) * (F.sigmoid_error(g) + 2.0**-21), "bf16")[:, fits])
