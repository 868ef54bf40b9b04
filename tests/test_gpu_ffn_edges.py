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
from .test_gpu_ffn import (LAYERS, MARK, SIZES, Layer, Step, bf, dev, f64, marked, near, out, rng,
                           run_product)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_required():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


TILES = 1 << 17  # rows expected that make any product take the tiles


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


@pytest.mark.parametrize("t,n,k", [(16, 72, 72), (64, 1032, 1032), (300, 520, 136)])
def test_lora_vanishing_inner_sums(t, n, k):
    """Inner sums down to the smallest binary32 numbers and below."""
    r = rng(t, n, 12)
    x, w = bf(r, t, k), bf(r, n, k)
    a, b = np.zeros((3, 8, k)), bf(r, 3, n, 8)
    a[:, np.arange(8), np.arange(8)] = 1
    scale, ad = 2.0 ** np.array([-100, -126, -146]), np.arange(t) % 4 - 1
    prm = mb.LoraParams.make(t, n, k, 8, 3, dtype_out="f32")
    y = out(t, n, dtype="f32")
    mb.project_lora(prm, dev(x), dev(w), dev(a), dev(b), dev(scale, torch.float32), ints(ad),
                    mb.alloc_lora_workspace(prm, G.dev()), y)
    want, err = F.lora(x, w, a, b, scale, ad)
    near(f64(y), want, F.rounded(want, err, "f32"))


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


def micros(call, calls=20):
    """Time of a call among others, the least of some runs."""
    best = float("inf")
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(calls):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / calls)
    return best


def test_empty_replica_slots_cost_little():
    """1024 replica slots without rows, against none (20 us; the search of every
    slot for every slot took 900)."""
    n = k = 64
    t = {}
    for R in (0, 16):
        L = Layer(np.pad(np.ones((64, 16), int), ((0, 0), (0, R))), 16)
        dy, a, dw = out(L.rows, n), out(L.rows, k), out(L.E, n, k)
        t[R] = micros(lambda: mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, dy, a, dw))
    assert t[16] < 5 * t[0], t


@pytest.mark.parametrize("t,n", [(4000, 8), (1000, 64), (240, 256)])
def test_lora_narrow_outputs_use_the_whole_gpu(t, n):
    """As many 16 x 16 tiles as CUs take little more than one (1.3 to 2.1 times;
    a workgroup to a column alone took 10 to 140)."""
    k, r = 7168, rng(t)
    took = {}
    for rows, cols in ((16, 16), (t, n)):
        prm = mb.LoraParams.make(rows, cols, k, 16, 2)
        x, w, a, b, y = out(rows, k), out(cols, k), out(2, 16, k), out(2, cols, 16), out(rows, cols)
        args = (x, w, a, b, torch.ones(2, device=G.dev()), ints(r.integers(0, 2, rows)),
                mb.alloc_lora_workspace(prm, G.dev()), y)
        took[rows] = micros(lambda: mb.project_lora(prm, *args))
    assert took[t] < 6 * took[16], took


def test_many_replicas_of_an_expert():
    """Every replica slot holds one of two experts, and every second has rows."""
    r = rng(21)
    counts = np.ones((64, 18), int)
    counts[:, 2:] = r.integers(0, 4, (64, 16)) * (np.arange(16) % 2)
    L = Layer(counts, 2, r.integers(0, 2, (64, 16)) * 77 + 50, pad=1)
    n, k = 40, 72
    dy, a, dw = bf(r, L.rows, n), bf(r, L.rows, k), out(L.E, n, k, dtype="f32")
    mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, L.tensor(dy), L.tensor(a), dw)
    got = f64(dw)
    for e in range(L.E):
        rows = np.concatenate([np.arange(lo, hi) for x, lo, hi in L.groups if x == e])
        v, err = F.weight_grad(dy[rows], a[rows])
        near(got[e], v, F.rounded(v, err, "f32"))


# ------------------------------------------------------------ tiles, and few rows

@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("layer", [name for name in LAYERS if name != "few"])
def test_products_in_tiles(layer, n, k):
    """Sizes that by themselves would take their operands straight from memory."""
    run_product(LAYERS[layer](expected=TILES), n, k, "none", "bf16")
    run_product(LAYERS[layer](expected=TILES, dtype_out="f32"), n, k, "none", "f32")
    run_product(LAYERS[layer](expected=TILES), n, k, "swiglu", "bf16")
    run_product(LAYERS[layer](expected=TILES), n, k, "swiglu", "bf16", keep=False)


@pytest.mark.parametrize("counts,home", [
    ([[9]], 1), ([[16]], 1), ([[17]], 1), ([[64]], 1), ([[129]], 1),
    ([[12], [0], [33], [5]], 1), ([[16, 16, 16, 16]], 4), ([[1, 140, 0, 3]], 3),
])
def test_products_of_few_rows_and_slots(counts, home):
    """On both sides of where the columns of tiles leave more than half the CUs
    idle: outputs of one column up to 130."""
    for n, k in ((264, 520), (4104, 264), (16648, 40)):
        run_product(Layer(counts, home, pad=1), n, k, "none", "bf16")
        run_product(Layer(counts, home, dtype_out="f32"), n, k, "none", "f32")
        run_product(Layer(counts, home), n, k, "swiglu", "bf16")


@pytest.mark.parametrize("expected", [2, TILES])
def test_infinities_stay_in_their_rows_and_columns(expected):
    L = Layer([[40, 3]], 2, expected=expected, dtype_out="f32")
    n, k = 24, 88
    r = rng(5, expected)
    a, w = bf(r, L.rows, k), bf(r, 2, n, k)
    a[7, 80], w[0, 5, 3], a[41, 0] = np.nan, np.inf, -np.inf
    y = out(L.rows, n, dtype="f32")
    mb.expert_bf16(L.dims, L.bufs, n, k, dev(a), dev(w), y)
    want = np.ones((L.rows, n), bool)
    want[7], want[:40, 5], want[41] = False, False, False
    assert np.array_equal(np.isfinite(f64(y)), want)


@pytest.mark.parametrize("expected", [2, TILES])
def test_products_under_a_fatal_status(expected):
    L = Layer([[37, 0, 5, 1], [0, 70, 13, 2]], 3, expected=expected)
    L.bufs.status[0] = mb.ST_CAPACITY
    y, pre = out(L.rows, 64), out(L.rows, 128)
    a, w = out(L.rows, 72), out(L.E, 128, 72)
    mb.expert_bf16(L.dims, L.bufs, 64, 72, a, w, y)
    mb.expert_bf16(L.dims, L.bufs, 64, 72, a, w, y, act="swiglu", pre=pre)
    assert marked(y).all() and marked(pre).all()


def test_a_slot_of_few_rows_takes_little_more_than_eight():
    """Nine rows in one slot are as many 16-row blocks as eight (1.0 times; in
    tiles, which leave nine CUs of ten idle, 3.2)."""
    h, i = 7168, 3200
    w, took = out(1, 2 * i, h), {}
    for rows in (8, 9, 16):
        L = Layer([[rows]], 1)
        a, y = out(rows, h), out(rows, i)
        took[rows] = micros(lambda: mb.expert_bf16(L.dims, L.bufs, i, h, a, w, y, act="swiglu"))
    assert max(took.values()) < 2 * took[8], took


def test_a_training_step_in_tiles():
    """As a_training_step, whose bounds these are, with rows enough for tiles in
    every product, captured and replayed."""
    s = Step(N=3000, H=1032, I=520, seed=9)
    s.run()
    for name, want in s.exact().items():
        want, got = want.detach().numpy(), f64(s.o[name])
        rms = np.sqrt((want**2).mean())
        near(got, want, 12 * 2.0**-8 * (rms + np.abs(want)))
    keep = {k: s.o[k].clone() for k in ("y", "dx", "dgate", "dw1", "dw2")}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        s.run(st)
    for _ in range(3):
        for v in s.o.values():
            v.fill_(MARK)
        g.replay()
        torch.cuda.synchronize()
        for k, v in keep.items():
            assert torch.equal(s.o[k], v), k


# ------------------------------------------------------------ far gates

@pytest.mark.parametrize("expected", [1, TILES])
@pytest.mark.parametrize("rows", [3, 64, 300])
def test_far_gates_of_large_ups_keep_their_value(rows, expected):
    """silu(g) u where silu(g) alone is below binary32 and u brings it back."""
    gates = np.array([-170, -150, -130, -110, -104, -95, -88.5, -81, -60, -3, 0.5, 90])
    ups = 2.0 ** np.array([0, 30, 60, 90, 120])
    n, k = len(gates) * len(ups) + 4, 8
    pair = np.array([(g, u) for g in gates for u in ups] + [(1, 1)] * 4)
    pair = R.bf16_round(np.float32(pair)).astype(np.float64)
    L = Layer([[rows]], 1, expected=expected)
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


# ------------------------------------------------------------ past 2^31 elements

def blank(*shape, dtype=torch.bfloat16):
    return torch.full(shape, MARK, dtype=dtype, device=G.dev())


def untouched(t, rows):
    """Whether all rows but these still hold the mark (in pieces: the tensors are large)."""
    keep = torch.ones(t.shape[0], dtype=torch.bool, device=t.device)
    keep[torch.from_numpy(rows).to(t.device)] = False
    mark = torch.tensor(MARK, dtype=t.dtype, device=t.device)
    return all(bool((p == mark).all(1)[k].all()) for p, k in zip(t.split(1 << 17), keep.split(1 << 17)))


def region(counts, cap, expected, home=1, dtype_out="bf16"):
    """A layer whose ranks' regions have `cap` rows, few of them used."""
    L = Layer(counts, home, pad=cap - int(np.asarray(counts).sum(axis=1).max()), expected=expected,
              dtype_out=dtype_out)
    assert L.cap == cap
    return L, np.flatnonzero(L.used)


@pytest.mark.parametrize("expected", [12, 3 << 17])  # operands straight from memory, tiles
def test_rows_past_two_billion_elements(expected):
    cap, n, k = 1 << 19, 2056, 72
    L, used = region([[5], [0], [37]], cap, expected)
    assert L.rows * n > 1 << 31
    r = rng(expected)
    at = torch.from_numpy(used).to(G.dev())
    thin, wide = bf(r, len(used), k), bf(r, len(used), n)
    a, y = blank(L.rows, k), blank(L.rows, n)
    a[at] = dev(thin)
    w = bf(r, L.E, n, k, std=k**-0.5)
    rows = {e: np.searchsorted(used, np.arange(lo, hi)) for e, lo, hi in L.groups}
    mb.expert_bf16(L.dims, L.bufs, n, k, a, dev(w), y)
    got = f64(y[at])
    for e, i in rows.items():
        v, err = F.product(thin[i], w[e])
        near(got[i], v, F.rounded(v, err, "bf16"))
    assert untouched(y, used)
    # long rows in, and the weights' gradient of both
    y[at] = dev(wide)
    da = blank(L.rows, k)
    mb.expert_bf16_dgrad(L.dims, L.bufs, n, k, y, dev(w), da)
    dw = out(L.E, n, k, dtype="f32")
    mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, y, a, dw)
    got = f64(da[at])
    for e, i in rows.items():
        v, err = F.row_grad(wide[i], w[e])
        near(got[i], v, F.rounded(v, err, "bf16"))
        v, err = F.weight_grad(wide[i], thin[i])
        near(f64(dw[e]), v, F.rounded(v, err, "f32"))
    assert untouched(da, used)
    dw = out(L.E, k, n, dtype="f32")
    mb.expert_bf16_wgrad(L.dims, L.bufs, k, n, a, y, dw)
    for e, i in rows.items():
        v, err = F.weight_grad(thin[i], wide[i])
        near(f64(dw[e]), v, F.rounded(v, err, "f32"))


@pytest.mark.parametrize("expected", [12, 3 << 17])
def test_gated_rows_past_two_billion_elements(expected):
    cap, n, k = 1 << 18, 1416, 72
    L, used = region([[5], [0], [37]], cap, expected)
    assert L.rows * 2 * n > 1 << 31
    r = rng(expected, 1)
    at = torch.from_numpy(used).to(G.dev())
    x, w = bf(r, len(used), k), bf(r, L.E, 2 * n, k, std=k**-0.5)
    a, y, pre = blank(L.rows, k), blank(L.rows, n), blank(L.rows, 2 * n)
    a[at] = dev(x)
    rows = {e: np.searchsorted(used, np.arange(lo, hi)) for e, lo, hi in L.groups}
    mb.expert_bf16(L.dims, L.bufs, n, k, a, dev(w), y, act="swiglu", pre=pre)
    got, gp = f64(y[at]), f64(pre[at])
    for e, i in rows.items():
        g, eg, u, eu, h, eh = F.gated(x[i], w[e])
        near(got[i], h, F.rounded(h, eh, "bf16"))
        near(gp[i], np.concatenate((g, u), 1), F.rounded(np.concatenate((g, u), 1),
                                                         np.concatenate((eg, eu), 1), "bf16"))
    assert untouched(y, used) and untouched(pre, used)
    dp, w2 = blank(L.rows, 2 * n), bf(r, L.E, k, n, std=k**-0.5)
    mb.expert_bf16_dgrad(L.dims, L.bufs, k, n, a, dev(w2), dp, act="swiglu", pre=pre)
    got = f64(dp[at])
    for e, i in rows.items():
        dg, eg, du, eu = F.gate_grad(x[i], w2[e], gp[i, :n], gp[i, n:])
        near(got[i, :n], dg, F.rounded(dg, eg, "bf16"))
        near(got[i, n:], du, F.rounded(du, eu, "bf16"))
    assert untouched(dp, used)


@pytest.mark.parametrize("expected", [64, TILES])
def test_weights_past_two_billion_elements(expected):
    """1024 experts; the first, one in the middle and the last have rows."""
    n, k = 2064, 1032  # (half of n is a multiple of 8 too)
    counts = np.zeros((64, 16), int)
    counts[0, 0], counts[31, 5], counts[63, 15] = 3, 40, 21
    r = rng(expected, 2)
    some = [0, 31 * 16 + 5, 1023]
    w = torch.full((1024, n, k), float("nan"), dtype=torch.bfloat16, device=G.dev())
    assert w.numel() > 1 << 31
    few = {e: bf(r, n, k, std=k**-0.5) for e in some}
    for e in some:
        w[e] = dev(few[e])
    L = Layer(counts, 16, expected=expected)
    a, dy = bf(r, L.rows, k), bf(r, L.rows, n)
    y, da, mid = out(L.rows, n), out(L.rows, k), out(L.rows, n // 2)
    mb.expert_bf16(L.dims, L.bufs, n, k, L.tensor(a), w, y)
    mb.expert_bf16(L.dims, L.bufs, n // 2, k, L.tensor(a), w, mid, act="swiglu")
    mb.expert_bf16_dgrad(L.dims, L.bufs, n, k, L.tensor(dy), w, da)
    for e, lo, hi in L.groups:
        v, err = F.product(a[lo:hi], few[e])
        near(f64(y[lo:hi]), v, F.rounded(v, err, "bf16"))
        _, _, _, _, v, err = F.gated(a[lo:hi], few[e])
        near(f64(mid[lo:hi]), v, F.rounded(v, err, "bf16"))
        v, err = F.row_grad(dy[lo:hi], few[e])
        near(f64(da[lo:hi]), v, F.rounded(v, err, "bf16"))
    del w
    dw = blank(1024, n, k, dtype=torch.float32)
    mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, L.tensor(dy), L.tensor(a), dw)
    rest = np.setdiff1d(np.arange(1024), some)
    assert not any(bool(p.any()) for p in dw[torch.from_numpy(rest).to(G.dev())].split(64))
    mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, L.tensor(dy), L.tensor(a), dw, accumulate=True)
    for e, lo, hi in L.groups:  # twice the sum, rounded in between
        v, err = F.weight_grad(dy[lo:hi], a[lo:hi])
        near(f64(dw[e]), 2 * v, 2 * F.rounded(v, err, "f32") + 2.0**-23 * np.abs(2 * v))


@pytest.mark.parametrize("n,k,h", [
    (300001, 1, 7168),     # both rows and tokens past 2^31 elements
    ((1 << 22) + 7, 1, 8), ((1 << 21) + 3, 2, 1024), ((1 << 20) + 3, 1, 1032),  # the launch goes round
])
def test_combine_gradients_of_many_tokens(n, k, h):
    g = torch.Generator(device=G.dev())
    g.manual_seed(n)
    d = mb.Dims.make(n, k, max(k, 2), 1, 0, h, cap=n * k + 3)
    bufs = mb.PlanBuffers.allocate(d, G.dev())
    bufs.pos = torch.randperm(n * k + 3, generator=g, device=G.dev())[: n * k].int().view(n, k)
    bufs.status.zero_()
    dy, ye = (torch.empty(m, h, dtype=torch.bfloat16, device=G.dev()).normal_(generator=g)
              for m in (n, d.rows))
    w = torch.rand(n, k, generator=g, device=G.dev())
    go, gw = blank(d.rows, h), blank(n, k, dtype=torch.float32)
    mb.combine_grad(d, bufs, dy, ye, w, go, gw)
    for lo in range(0, n, 1 << 17):
        t = slice(lo, min(lo + (1 << 17), n))
        for j in range(k):
            at = bufs.pos[t, j].long()
            # one product in binary32, rounded once: the same bits
            assert torch.equal(go[at], (w[t, j:j + 1] * dy[t].float()).bfloat16())
            prod = dy[t].double() * ye[at].double()
            err = (gw[t, j].double() - prod.sum(1)).abs()
            bound = (h * F.ADD + F.STEP["f32"]) * prod.abs().sum(1) + F.TINY
            assert bool((err <= bound).all())
    rest = torch.ones(d.rows, dtype=torch.bool, device=G.dev())
    rest[bufs.pos.view(-1).long()] = False
    assert bool((go[rest] == torch.tensor(MARK, dtype=go.dtype, device=go.device)).all())


@pytest.mark.parametrize("t,n,k,rank,L", [
    ((1 << 19) + 600, 4104, 8, 8, 2), ((1 << 19) + 600, 8, 4104, 8, 2),  # outputs, rows
    ((1 << 23) + 100, 8, 8, 256, 2),                                     # the inner sums
    (5, 8200, 8, 256, 1024), (300, 8200, 8, 256, 1024),                  # the adapters
    (5, 8, 8200, 256, 1024), (300, 264, 8200, 256, 1024),
])
def test_lora_past_two_billion_elements(t, n, k, rank, L):
    g = torch.Generator(device=G.dev())
    g.manual_seed(t + n)
    r = rng(t, n)

    def rows(m, c):
        return torch.empty(m, c, dtype=torch.bfloat16, device=G.dev()).normal_(generator=g)

    x, w, a, b = rows(t, k), rows(n, k), rows(L * rank, k), rows(L * n, rank)
    assert max(t * n, t * k, t * rank, L * n * rank, L * rank * k) > 1 << 31
    ad = np.sort(r.integers(-1, L, t))
    ad[-1] = L - 1
    prm = mb.LoraParams.make(t, n, k, rank, L)
    y = blank(t, n)
    mb.project_lora(prm, x, w, a.view(L, rank, k), b.view(L, n, rank),
                    torch.ones(L, device=G.dev()), ints(ad), mb.alloc_lora_workspace(prm, G.dev()), y)
    for i in np.unique(np.concatenate((np.arange(min(t, 5)), r.integers(0, t, 12), t - 1 - np.arange(5)))):
        e = ad[i]
        low = (f64(a[e * rank:(e + 1) * rank])[None], f64(b[e * n:(e + 1) * n])[None]) if e >= 0 else (
            np.zeros((1, rank, k)), np.zeros((1, n, rank)))
        want, err = F.lora(f64(x[i:i + 1]), f64(w), *low, np.ones(1), [0])
        near(f64(y[i:i + 1]), want, F.rounded(want, err, "bf16"))


@pytest.mark.parametrize("expected", [1, TILES])
def test_the_widest_outputs_and_longest_sums(expected):
    """2^20 outputs, and sums of 2^20 terms, of one slot with a tile and a rest."""
    wide, k, rows = 1 << 20, 8, 70
    L = Layer([[rows]], 1, pad=1, expected=expected, dtype_out="f32")
    r = rng(expected, 7)
    a, w = bf(r, L.rows, k), bf(r, 1, wide, k)
    y = out(L.rows, wide, dtype="f32")
    mb.expert_bf16(L.dims, L.bufs, wide, k, L.tensor(a), dev(w), y)
    v, err = F.product(a[:rows], w[0])
    near(f64(y[:rows]), v, F.rounded(v, err, "f32"))
    assert marked(y[rows:]).all()
    half = wide // 2
    mid, pre = out(L.rows, half), out(L.rows, wide)
    mb.expert_bf16(L.dims, L.bufs, half, k, L.tensor(a), dev(w), mid, act="swiglu", pre=pre)
    g, eg, u, eu, h, eh = F.gated(a[:rows], w[0])
    near(f64(mid[:rows]), h, F.rounded(h, eh, "bf16"))
    near(f64(pre[:rows, :half]), g, F.rounded(g, eg, "bf16"))
    near(f64(pre[:rows, half:]), u, F.rounded(u, eu, "bf16"))
    # the gradient of the rows: sums of 2^20 terms, then 2^20 of them
    dy = bf(r, L.rows, wide, std=2.0**-10)
    da = out(L.rows, k, dtype="f32")
    mb.expert_bf16_dgrad(L.dims, L.bufs, wide, k, L.tensor(dy), dev(w), da)
    v, err = F.row_grad(dy[:rows], w[0])
    near(f64(da[:rows]), v, F.rounded(v, err, "f32"))
    w2, p = bf(r, 1, k, half), f64(pre)[:rows]
    dp = out(L.rows, wide)
    mb.expert_bf16_dgrad(L.dims, L.bufs, k, half, L.tensor(a), dev(w2), dp, act="swiglu", pre=pre)
    dg, eg, du, eu = F.gate_grad(a[:rows], w2[0], p[:, :half], p[:, half:])
    near(f64(dp[:rows, :half]), dg, F.rounded(dg, eg, "bf16"))
    near(f64(dp[:rows, half:]), du, F.rounded(du, eu, "bf16"))
    for one, two in ((dy, a), (a, dy)):
        dw = out(1, one.shape[1], two.shape[1], dtype="f32")
        mb.expert_bf16_wgrad(L.dims, L.bufs, one.shape[1], two.shape[1], L.tensor(one), L.tensor(two), dw)
        v, err = F.weight_grad(one[:rows], two[:rows])
        near(f64(dw[0]), v, F.rounded(v, err, "f32"))


@pytest.mark.parametrize("t,n,k", [(5, 1 << 20, 8), (70, 1 << 20, 8), (5, 8, 1 << 20), (70, 8, 1 << 20),
                                   (300, 264, 1 << 18), (1 << 26, 8, 8)])
def test_lora_of_the_largest_sizes(t, n, k):
    g = torch.Generator(device=G.dev())
    g.manual_seed(t + n)

    def rows(m, c, std=1.0):
        return torch.empty(m, c, dtype=torch.bfloat16, device=G.dev()).normal_(0, std, generator=g)

    x, w, a, b = rows(t, k), rows(n, k, k**-0.5), rows(16, k, k**-0.5), rows(2 * n, 8)
    ad = torch.randint(-1, 2, (t,), generator=g, device=G.dev(), dtype=torch.int32)
    prm = mb.LoraParams.make(t, n, k, 8, 2, dtype_out="f32")
    y = blank(t, n, dtype=torch.float32)
    mb.project_lora(prm, x, w, a.view(2, 8, k), b.view(2, n, 8), torch.ones(2, device=G.dev()), ad,
                    mb.alloc_lora_workspace(prm, G.dev()), y)
    some = np.unique(np.concatenate((np.arange(min(t, 9)), t - 1 - np.arange(5), rng(t).integers(0, t, 9))))
    at = torch.from_numpy(some).to(G.dev())
    want, err = F.lora(f64(x[at]), f64(w), f64(a).reshape(2, 8, k), f64(b).reshape(2, n, 8), np.ones(2),
                       ad[at].tolist())
    near(f64(y[at]), want, F.rounded(want, err, "f32"))
    assert bool((y != MARK).any(1).all())
