"""The router, the norm, the 4-bit rows and the experts' products on the GPU
against their plain 64-bit definitions (``plain_ops``).

Tolerances, derived from the arithmetic before any run:

* route: ids exact. Weights are binary32: an exponential (argument reduction
  and result, at most 4 * 2^-24 relative for the chosen ones), a sum of at
  most 1024 terms added in a tree with at most 64 of them in line (80 roundings
  of 2^-24), a division and the scale: below 2^-17 relative.
* norm: the sum of H squares adds at most 72 terms in line in binary32 and the
  root halves its error; with the products after it: below 2^-18 relative on
  scales and normed values. The codes are the values within half a step of
  e4m3 (2^-4 relative, 2^-10 scales for subnormal codes) and that error.
* 4-bit rows: scales by powers of two are exact, so codes and scale bytes are
  equal; after the activation (binary32 exponential, division and products:
  below 2^-18 relative) a value may round to the other side of a midpoint
  that it is that close to.
* experts: the products of two elements are exact, their sum is taken in
  binary32 in an order of the matrix unit's own: each of the k additions may
  be off by 2^-23 of the sum of magnitudes; bf16 outputs half a step, 2^-8.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import token_dispatch_mb_amd as mb
import workload as W

from . import gpu_harness as G
from . import plain_ops as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu_required():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(G.dev())


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def rng(*seed):
    return np.random.default_rng(seed)


# ------------------------------------------------------------------- route

def check_route(l, dtype, k, bias=None, **kw):
    l = np.asarray(l, np.float32)
    if dtype == "bf16":
        l = R.bf16_round(l)
    n, e = l.shape
    prm = mb.RouteParams.make(n, e, k, dtype=dtype, **kw)
    ids = torch.full((n, k), -7, dtype=torch.int32, device=G.dev())
    w = torch.full((n, k), float("nan"), device=G.dev())
    b = None if bias is None else dev(np.asarray(bias, np.float32))
    mb.route(prm, dev(l, DT[dtype]), ids, w, bias=b)
    want, ww = R.route(l, k, bias=None if bias is None else np.asarray(bias, np.float32), **kw)
    got = ids.cpu().numpy()
    bad = np.nonzero((got != want).any(axis=1))[0]
    assert not len(bad), (len(bad), bad[:5], got[bad[:3]], want[bad[:3]])
    gw = f64(w)
    assert np.all(np.abs(gw - ww) <= 2.0**-17 * np.abs(ww) + 1e-37), np.abs(gw - ww).max()
    return got, gw


ROUTES = [  # N, E, K, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (77, 8, 2, 1, 1, 1), (65, 16, 4, 4, 2, 2),
    (301, 60, 4, 1, 1, 1), (301, 64, 6, 8, 3, 1), (130, 100, 10, 4, 2, 2), (130, 128, 8, 1, 1, 1),
    (258, 160, 6, 8, 3, 1), (1031, 256, 8, 8, 4, 2), (513, 256, 8, 1, 1, 1), (203, 384, 8, 1, 1, 1),
    (203, 384, 8, 8, 4, 2), (99, 320, 9, 16, 5, 2), (40, 512, 16, 64, 9, 2), (33, 1024, 32, 1, 1, 1),
    (33, 1024, 32, 2, 1, 2), (5, 999, 7, 3, 2, 1), (70, 512, 8, 8, 4, 2), (70, 512, 14, 1, 1, 1),
    (70, 512, 15, 1, 1, 1), (41, 128, 8, 8, 4, 2), (41, 64, 8, 16, 8, 2), (41, 256, 8, 2, 1, 1),
    (41, 256, 8, 4, 2, 2), (41, 384, 8, 16, 3, 2), (41, 200, 8, 1, 1, 1), (41, 48, 8, 1, 1, 1),
    (41, 130, 8, 1, 1, 1), (41, 16, 14, 1, 1, 1), (41, 16, 16, 1, 1, 1),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,e,k,g,tg,gt", ROUTES)
def test_route(n, e, k, g, tg, gt, score):
    r = rng(n, e, k)
    l = 2 * r.standard_normal((n, e))
    bias = 0.1 * r.standard_normal(e)
    kw = dict(score=score, n_groups=g, top_groups=tg, group_top=gt)
    check_route(l, "f32", k, bias=bias, scale=2.5, **kw)
    check_route(l, "bf16", k, bias=bias, renorm=False, **kw)
    check_route(l, "f32", k, renorm=False, **kw)
    check_route(l, "bf16", k, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,g,tg,gt", [(16, 4, 1, 1, 1), (256, 8, 8, 4, 2), (60, 5, 1, 1, 1),
                                         (384, 8, 1, 1, 1), (256, 8, 8, 4, 1)])
def test_route_rows_out_of_the_ordinary(e, k, g, tg, gt, score):
    """Ties, masks, infinities, NaN, values a rounding apart, far logits."""
    r = rng(e, k)
    n = 24
    l = r.standard_normal((n, e)).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2] = 1.25
    l[3, : e // 2] = -np.inf
    l[4, 1:] = -np.inf
    l[5, [3, e - 2]] = np.inf
    l[6, ::2] = np.nan
    l[7] = -200 - np.arange(e)  # every score underflows in binary32
    l[8] = 20 + np.arange(e) * 2e-6  # sigmoids a rounding apart
    l[9] = np.float32(0.5) + np.arange(e)[::-1] * np.float32(2.0**-24)
    l[10] = np.round(l[10])
    l[11] = 80 * l[11]
    l[12, ::3] = l[12, 0]
    l[13] = 0.0
    l[13, 1::2] = -0.0
    l[14] = np.float32(-3e38)
    l[15] = np.float32(3e38)
    l[16, 5] = np.float32(3.4e38)
    l[17] = 1e-40 * np.arange(e)
    l[18, :-1] = -np.inf
    l[19] = np.where(np.arange(e) < k - 1, l[19], -np.inf)
    l[20] = np.where(np.arange(e) % 5 == 0, np.inf, np.nan)
    kw = dict(score=score, n_groups=g, top_groups=tg, group_top=gt)
    bias = (0.1 * r.standard_normal(e)).astype(np.float32)
    odd = bias.copy()
    odd[0], odd[5], odd[7], odd[e - 1] = -np.inf, np.nan, np.inf, -np.inf
    for dtype in ("f32", "bf16"):
        for renorm in (True, False):
            for b in (None, bias, np.zeros(e, np.float32), odd, np.full(e, -np.inf, np.float32)):
                check_route(l, dtype, k, bias=b, renorm=renorm, **kw)


def test_route_many_tokens_near_borders():
    """Quantised biases and logits: many choice values within a few roundings
    of each other, and many equal."""
    r = rng(5)
    l = np.round(r.standard_normal((4000, 256)) * 8) / 8
    bias = np.round(r.standard_normal(256) * 4) / 64
    l[2000:] = np.round(l[2000:]) + 2.0**-20 * r.integers(0, 3, (2000, 256))
    check_route(l, "f32", 8, bias=bias, score="sigmoid", n_groups=8, top_groups=4, group_top=2)
    check_route(l, "f32", 8, bias=0 * bias, score="softmax")
    check_route(l, "bf16", 8, score="softmax")
    check_route(l, "f32", 8, score="sigmoid")


def test_route_without_tokens_and_tail_untouched():
    prm = mb.RouteParams.make(3, 64, 4)
    ids = torch.full((5, 4), -7, dtype=torch.int32, device=G.dev())
    w = torch.full((5, 4), 9.0, device=G.dev())
    l = torch.randn(5, 64, device=G.dev())
    mb.route(mb.RouteParams.make(0, 64, 4), l, ids, w)
    assert (ids == -7).all() and (w == 9).all()
    mb.route(prm, l, ids, w)
    assert (ids[3:] == -7).all() and (w[3:] == 9).all() and (ids[:3] >= 0).all()


# -------------------------------------------------------------------- norm

def check_norm(x, weight, eps, dtype, residual=None, in_place=None, want_y=True):
    d = DT[dtype]
    cast = (lambda a: a) if dtype == "f32" else R.bf16_round
    x, weight = cast(np.float32(x)), cast(np.float32(weight))
    res = None if residual is None else cast(np.float32(residual))
    n, h = x.shape
    xd, wd = dev(x, d), dev(weight, d)
    rd = None if res is None else dev(res, d)
    out = None
    if res is not None:
        out = {"x": xd, "residual": rd}.get(in_place)
        out = torch.empty_like(xd) if out is None else out
    y = torch.empty_like(xd) if want_y else None
    q = torch.full((n, h), 0xA5, dtype=torch.uint8, device=G.dev())
    qs = torch.full((n, h // 128), -5.0, device=G.dev())
    mb.rmsnorm_fp8(xd, wd, eps, q, qs, residual=rd, residual_out=out, y=y)
    hh = x if res is None else x + res  # binary32, as the kernel's
    if res is not None:
        want = hh if dtype == "f32" else R.bf16_round(hh)
        assert np.array_equal(out.float().cpu().numpy(), want, equal_nan=True)
    ss = (hh.astype(np.float64) ** 2).sum(axis=1)
    bad = ~(ss < 3.4e38)
    _, yy, scale = R.rmsnorm(x, weight, eps, res)
    gq, gs = q.cpu().numpy(), f64(qs)
    assert np.isnan(gs[bad]).all() and (gq[bad] & 0x7F == 0x7F).all()
    yy, scale, gq, gs = yy[~bad], scale[~bad], gq[~bad], gs[~bad]
    assert np.all(np.abs(gs - scale) <= 2.0**-18 * scale), np.abs(gs / scale - 1).max()
    v = R.e4m3_values(gq) * np.repeat(gs, 128, axis=1)
    # blocks whose scale is far below a normal binary32 are zeros
    tol = np.maximum(2.0**-4 * np.abs(yy), 2.0**-10 * np.repeat(scale, 128, axis=1)) * (
        1 + 2.0**-16) + 2.0**-17 * np.abs(yy) + 2.0**-110
    assert np.all(np.abs(v - yy) <= tol), (np.abs(v - yy) / tol).max()
    if want_y:
        gy = f64(y)
        assert np.isnan(gy[bad]).all()
        half = 2.0**-24 if dtype == "f32" else 2.0**-8
        assert np.all(np.abs(gy[~bad] - yy) <= (half + 2.0**-18) * np.abs(yy) + 2.0**-126)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,h", [(1, 128), (3, 256), (1, 7168), (77, 384), (5, 1152), (9, 2048),
                                 (130, 4224), (33, 7168), (4, 8192), (3, 16384), (1025, 128)])
def test_norm(n, h, dtype):
    r = rng(n, h)
    x = r.standard_normal((n, h)) * np.exp(2 * r.standard_normal((n, 1)))
    res = 3 * r.standard_normal((n, h))
    w = 1 + 0.2 * r.standard_normal(h)
    check_norm(x, w, 1e-6, dtype)
    check_norm(x, w, 1e-6, dtype, want_y=False)
    check_norm(x, w, 1e-5, dtype, residual=res)
    check_norm(x, w, 1e-5, dtype, residual=res, in_place="x", want_y=False)
    check_norm(x, w, 0.0, dtype, residual=res, in_place="residual")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("h", [256, 7168])
def test_norm_rows_out_of_the_ordinary(h, dtype):
    r = rng(h)
    x = r.standard_normal((14, h))
    x[0] = 0
    x[1, 7] = np.nan
    x[2, h - 1] = np.inf
    x[3, 0] = -np.inf
    x[4] = 1e20  # its squares pass binary32
    x[5] *= 1e-18
    x[6] *= 1e-30  # its squares vanish beside eps
    x[7, :128] = 0
    x[8] = 0
    x[8, 3] = 1e4
    x[9] *= 1e15
    w = 1 + 0.1 * r.standard_normal(h)
    w[128:160] = 0
    check_norm(x, w, 1e-6, dtype)
    check_norm(x, w, 1e-6, dtype, residual=r.standard_normal((14, h)))
    wz = w.copy()
    wz[128:256] = 1e-37
    check_norm(x, wz, 1e-6, dtype)
    check_norm(np.zeros((2, h)), w, 0.0, dtype)


def test_norm_refuses_overlaps():
    x = torch.randn(4, 256, device=G.dev())
    q = torch.empty(4, 256, dtype=torch.uint8, device=G.dev())
    qs = torch.empty(4, 2, device=G.dev())
    w = torch.ones(256, device=G.dev())
    with pytest.raises(ValueError, match="overlap"):
        mb.rmsnorm_fp8(x, w, 1e-6, q, qs, y=x)
    with pytest.raises(ValueError, match="overlap"):
        mb.rmsnorm_fp8(x[:3], w, 1e-6, q, qs, residual=x[:3], residual_out=x[1:])
    with pytest.raises(ValueError, match="overlap"):
        mb.rmsnorm_fp8(x, w, 1e-6, q, qs, residual=x.clone(), residual_out=x, y=x)
    with pytest.raises(ValueError, match="overlap"):
        mb.rmsnorm_fp8(x, w, 1e-6, x.view(torch.uint8), qs)
    with pytest.raises(ValueError, match="overlap"):
        mb.rmsnorm_fp8(x, x[1], 1e-6, q, qs, residual=x.clone(), residual_out=x)
    with pytest.raises(ValueError, match="overlap"):
        mb.rmsnorm_fp8(x, w, 1e-6, q, q.view(torch.float32))
    one = x.clone()  # x as its own residual, in place: doubled
    mb.rmsnorm_fp8(one, w, 1e-6, q, qs, residual=one, residual_out=one)
    assert torch.equal(one, 2 * x)
    with pytest.raises(ValueError, match="two dimensions"):
        mb.rmsnorm_fp8(x[0], w, 1e-6, q, qs)
    with pytest.raises(TypeError, match="weight must be"):
        mb.rmsnorm_fp8(x, w.bfloat16(), 1e-6, q, qs)
    with pytest.raises(ValueError, match="q_scale holds"):
        mb.rmsnorm_fp8(x, w, 1e-6, q, qs[:3])


# -------------------------------------------------------------- 4-bit rows

def quantize(x, dtype, act="none", row_src=None, fill=0xA5):
    m, h = x.shape
    h //= 2 if act == "swiglu" else 1
    q = torch.full((m, h // 2), fill, dtype=torch.uint8, device=G.dev())
    s = torch.full((m, h // 32), fill, dtype=torch.uint8, device=G.dev())
    mb.quantize_mx4(dev(np.float32(x), DT[dtype]), q, s, act=act, row_src=row_src)
    return q, s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,h", [(1, 32), (1, 7168), (3, 96), (77, 1152), (5, 544), (1030, 64),
                                 (9, 7168)])
def test_quantize_and_back(m, h, dtype):
    r = rng(m, h)
    x = r.standard_normal((m, h)) * np.exp(3 * r.standard_normal((m, 1)))
    x = np.float32(x) if dtype == "f32" else R.bf16_round(np.float32(x))
    q, s = quantize(x, dtype)
    ws = R.mx4_scale_bytes(np.float64(x))
    wq = R.pack4(R.mx4_codes(np.float64(x), ws))
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)
    back = torch.full((m, h), -9.0, dtype=DT[dtype], device=G.dev())
    mb.dequantize_mx4(q, s, back)
    assert np.array_equal(f64(back), R.mx4_values(wq, ws))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_values_out_of_the_ordinary(dtype):
    """Every midpoint and magnitude at several scales, zeros of both signs,
    denormals, the largest finite values, infinities and NaN."""
    r = rng(1)
    grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.75])
    rows = []
    for ex in (0, 5, -7, 60, -60, 125, -126, -133, 90):
        b = np.zeros(32)
        b[:17] = grid
        b[17:30] = -grid[:13]
        b[30:] = [-0.0, 7.0]
        rows.append(b * 2.0 ** ex if ex < 125 else np.minimum(b * 2.0**125, 3.38e38))
    rows.append(np.zeros(32))
    rows.append(-np.zeros(32))
    for bad in (np.nan, np.inf, -np.inf):
        b = r.standard_normal(32)
        b[r.integers(32)] = bad
        rows.append(b)
    rows.append(np.full(32, 1e-45))
    rows.append(np.full(32, 1.5e-39))
    rows.append(np.full(32, 3.3e38))
    rows.append(np.nextafter(np.float32(8.0), np.float32(0)) * np.ones(32))
    with np.errstate(over="ignore"):
        x = np.float32(np.stack(rows))
    x = x if dtype == "f32" else R.bf16_round(x)
    q, s = quantize(x, dtype)
    ws = R.mx4_scale_bytes(np.float64(x))
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), R.pack4(R.mx4_codes(np.float64(x), ws)))
    back = torch.empty(x.shape, dtype=DT[dtype], device=G.dev())
    mb.dequantize_mx4(q, s, back)
    assert np.array_equal(f64(back), R.mx4_values(q.cpu().numpy(), ws), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_dequantize_every_code_and_scale(dtype):
    q = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1))
    s = np.repeat(np.arange(256, dtype=np.uint8), 16)[:, None]
    out = torch.empty(len(q), 32, dtype=DT[dtype], device=G.dev())
    mb.dequantize_mx4(dev(q), dev(s), out)
    want = R.mx4_values(q, s)
    with np.errstate(over="ignore"):
        want = np.float32(want).astype(np.float64)  # 6 * 2^127 passes binary32: infinite
    assert np.array_equal(f64(out), want, equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,h", [(1, 32), (130, 2048), (7, 96)])
def test_swiglu_quantize(m, h, dtype):
    r = rng(m, h, 2)
    x = np.float32(3 * r.standard_normal((m, 2 * h)))
    x = x if dtype == "f32" else R.bf16_round(x)
    x[0, 0], x[0, h] = -95.0, 2.0  # exp(95) is finite, the product tiny
    v = R.swiglu(x)
    q, s = quantize(x, dtype, act="swiglu")
    s = s.cpu().numpy()
    near = R.mx4_scale_bytes(v * (1 - 2.0**-17)), R.mx4_scale_bytes(v * (1 + 2.0**-17))
    assert ((s == near[0]) | (s == near[1])).all()
    unit = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, axis=1)
    got = R.mx4_values(q.cpu().numpy(), s)
    a = np.abs(v) / unit
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0)) * unit
    want = np.clip(v, -6 * unit, 6 * unit)
    assert np.all(np.abs(got - want) <= half + 2.0**-17 * np.abs(v)), np.abs(got - want).max()


def test_swiglu_of_far_gates():
    """Gates past the range of exp: silu(-200) is 0, silu(200) the gate."""
    x = np.zeros((1, 64))
    x[0, :32] = np.resize([-200.0, 200.0, -1e30, 1e30], 32)
    x[0, 32:] = 1.0
    q, s = quantize(x, "f32", act="swiglu")
    v = R.swiglu(x)
    assert np.array_equal(s.cpu().numpy(), R.mx4_scale_bytes(v))
    assert np.array_equal(np.abs(R.mx4_values(q.cpu().numpy(), s.cpu().numpy())),
                          np.abs(R.mx4_values(R.pack4(R.mx4_codes(v, s.cpu().numpy())),
                                              s.cpu().numpy())))


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_quantize_leaves_padding_rows(act):
    r = rng(9)
    x = np.float32(r.standard_normal((40, 256)))
    src = np.where(r.random(40) < 0.4, -1, np.arange(40)).astype(np.int32)
    q, s = quantize(x, "f32", act=act, row_src=dev(src))
    full, fs = quantize(x, "f32", act=act)
    keep = torch.from_numpy(src >= 0).to(G.dev())
    assert torch.equal(q[keep], full[keep]) and torch.equal(s[keep], fs[keep])
    assert (q[~keep] == 0xA5).all() and (s[~keep] == 0xA5).all()


# ----------------------------------------------------------------- experts

def make_plan(r, P, Eh, R_, cap, fill=0.8, empty=0.3):
    """cu_seqlens and rep_expert of a plan: skewed slots, some without rows,
    replicas of other ranks' experts or none."""
    E, ns = P * Eh, Eh + R_
    share = r.random((P, ns)) ** 3 * (r.random((P, ns)) > empty)
    rep = r.integers(0, E, (P, max(R_, 1))).astype(np.int32)
    rep[r.random(rep.shape) < 0.3] = -1
    if R_:
        share[:, Eh:][rep < 0] = 0
    tot = np.maximum(share.sum(axis=1, keepdims=True), 1e-9)
    n = np.floor(share / tot * cap * fill).astype(int)
    cu = np.zeros((P, ns + 1), np.int32)
    cu[:, 1:] = np.cumsum(n, axis=1)
    return cu, rep


class Product:
    """Random operands of the experts' products under a plan, on both sides."""

    def __init__(self, seed, P, Eh, R_, cap, n, k, out="bf16", tokens=None, plan=None, **kw):
        r = rng(seed, P, n, k)
        self.cu, self.rep = plan if plan else make_plan(r, P, Eh, R_, cap, **kw)
        E, rows = P * Eh, P * cap
        tokens = rows if tokens is None else tokens
        self.dims = mb.Dims.make(tokens, 1, E, P, R_, 128, cap=cap, dtype_out=out)
        self.n, self.k = n, k
        self.a, self.w = (r.integers(0, 256, (m, k // 2), dtype=np.uint8) for m in (rows, E * n))
        self.a_s, self.w_s = (r.integers(lo, lo + 6, (m, k // 32), dtype=np.uint8)
                              for lo, m in ((124, rows), (118, E * n)))
        self.groups = R.slots(self.cu, self.rep, P, Eh, R_, cap)
        self.bufs = mb.PlanBuffers.allocate(self.dims, G.dev())
        self.bufs.cu_seqlens.copy_(torch.from_numpy(self.cu))
        self.bufs.rep_expert.copy_(torch.from_numpy(self.rep))
        self.bufs.status.zero_()
        self.dev = [dev(t) for t in (self.a, self.a_s, self.w, self.w_s)]

    def out(self):
        return torch.full((self.dims.rows, self.n), -77.0, device=G.dev(),
                          dtype=G.out_dtype(self.dims))

    def run(self, y=None, stream=None):
        y = self.out() if y is None else y
        mb.expert_mx4(self.dims, self.bufs, self.n, self.k, *self.dev, y, stream=stream)
        return y

    def check(self, y):
        a, w = R.mx4_values(self.a, self.a_s), R.mx4_values(self.w, self.w_s)
        want, mag, used = R.expert(a, w.reshape(self.dims.n_experts, self.n, self.k), self.groups,
                                   self.n)
        got = f64(y)
        assert (got[~used] == -77).all(), "rows outside every slot were written"
        half = 2.0**-24 if self.dims.dtype_out == mb.F32 else 2.0**-8
        tol = self.k * 2.0**-23 * mag + half * np.abs(want) + 1e-30
        err = np.abs(got - want)[used]
        assert np.all(err <= tol[used]), (err / tol[used]).max()


EXPERTS = [  # P, Eh, R, cap, n, k
    (1, 1, 0, 1, 8, 128), (1, 1, 0, 300, 64, 128), (1, 8, 0, 40, 72, 256), (2, 2, 1, 33, 200, 384),
    (4, 4, 2, 17, 264, 512), (8, 1, 1, 130, 128, 640), (4, 2, 1, 520, 512, 1024),
    (2, 1, 0, 1000, 1032, 896), (64, 4, 1, 8, 256, 1152), (16, 24, 2, 12, 136, 256),
    (1, 2, 1, 2500, 296, 2048), (2, 4, 1, 64, 2048, 7168),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("P,Eh,R_,cap,n,k", EXPERTS)
def test_expert(P, Eh, R_, cap, n, k, out):
    p = Product(3, P, Eh, R_, cap, n, k, out)
    p.check(p.run())


@pytest.mark.parametrize("tokens", [1, 64, 600, 20000, 1 << 20])
def test_expert_any_expected_rows(tokens):
    """N*K only says how many rows to expect: whatever it is, every row of
    every slot is computed."""
    p = Product(4, 1, 5, 1, 700, 272, 512, tokens=tokens)
    p.check(p.run())


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 256, 257])
def test_expert_slot_sizes(rows):
    """Slots of one size, so that a tile ends at, before and behind its rows,
    with every tile size that an expected number of rows picks."""
    P, Eh, cap = 2, 2, 2 * rows + 3
    cu = np.array([[0, rows, 2 * rows], [0, 0, rows]], np.int32)
    for tokens in (2, 60, 200, 1 << 20):
        for k in (384, 512, 640, 1152):
            p = Product(rows, P, Eh, 0, cap, 160, k, tokens=tokens,
                        plan=(cu, np.full((P, 1), -1, np.int32)))
            p.check(p.run())


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 248, 256, 264, 520, 2056])
def test_expert_output_sizes(n, out):
    """Outputs that end inside a tile, in every kernel."""
    for tokens in (2, 60, 200, 1 << 20):
        p = Product(n, 2, 3, 1, 300, n, 512, out, tokens=tokens)
        p.check(p.run())


def test_expert_many_tiles_on_each_workgroup():
    """More tiles than workgroups, odd and even numbers of steps: rows and
    weights of the next tile are read under the last steps of one."""
    for k in (512, 640, 768, 896):
        p = Product(k, 8, 6, 1, 1500, 1288, k, tokens=1 << 20)
        p.check(p.run())


def test_expert_identity_layout():
    """One-hot rows against a weight per expert and column pin the operands'
    lane layout and the scales: y[p][j] = w[e][j][i(p)] * 2^s."""
    k, n, cap = 512, 48, 512
    cu = np.array([[0, cap]], np.int32)
    p = Product(1, 1, 1, 0, cap, n, k, "f32", plan=(cu, np.full((1, 1), -1, np.int32)))
    codes = np.zeros((cap, k), np.uint8)
    codes[np.arange(cap), np.arange(cap)] = 2  # 1.0 at element p of row p
    p.a = R.pack4(codes)
    p.a_s = np.tile((120 + np.arange(16)).astype(np.uint8), (cap, 1))
    p.dev[0], p.dev[1] = dev(p.a), dev(p.a_s)
    w = R.mx4_values(p.w, p.w_s)
    want = w.T * 2.0 ** (np.repeat(np.arange(16), 32) - 7.0)[:, None]
    assert np.array_equal(f64(p.run()), want)


def test_expert_nan_scale_stays_in_its_row():
    p = Product(6, 2, 2, 0, 40, 64, 256, "f32", empty=0.0)
    row = p.groups[0][1]
    p.a_s[row, 3] = 255
    p.dev[1] = dev(p.a_s)
    y = f64(p.run())
    assert np.isnan(y[row]).all()
    used = np.zeros(len(y), bool)
    for _, lo, hi in p.groups:
        used[lo:hi] = True
    used[row] = False
    assert np.isfinite(y[used]).all()
    # a NaN weight column reaches that output of its expert's rows only
    p = Product(6, 2, 2, 0, 40, 64, 256, "f32", empty=0.0)
    e, lo, hi = p.groups[1]
    p.w_s[e * 64 + 5, 7] = 255
    p.dev[3] = dev(p.w_s)
    y = f64(p.run())
    assert np.isnan(y[lo:hi, 5]).all()
    y[:, 5] = 0
    assert np.isfinite(y).all()


def test_expert_does_nothing_under_a_fatal_status():
    p = Product(7, 2, 2, 1, 40, 64, 256)
    for flag in (mb.ST_BAD_ID, mb.ST_DUP_ID, mb.ST_CAPACITY):
        p.bufs.status[0] = flag
        assert (p.run() == -77).all()
    p.bufs.status[0] = mb.ST_UNBALANCED
    p.check(p.run())


def test_expert_plan_out_of_range_stays_inside():
    """Offsets outside the region and experts outside [0, E) are cut to the
    buffer or left out."""
    P, Eh, R_, cap, n, k = 2, 1, 1, 50, 32, 128
    cu = np.array([[0, 30, 90], [-5, 20, 10]], np.int32)
    rep = np.array([[5], [-3]], np.int32)
    p = Product(8, P, Eh, R_, cap, n, k, plan=(cu, rep))
    p.groups = [(0, 0, 30), (1, 50, 70)]
    p.check(p.run())
    p.bufs.rep_expert.copy_(torch.from_numpy(np.array([[1], [0]], np.int32)))
    p.groups = [(0, 0, 30), (1, 30, 50), (1, 50, 70)]
    p.check(p.run())


def test_expert_two_streams_at_once():
    """Calls on two streams share nothing."""
    a = Product(10, 2, 4, 1, 400, 256, 512)
    b = Product(11, 8, 1, 1, 60, 384, 256, "f32")
    ya, yb = a.out(), b.out()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(ya, s1)
        b.run(yb, s2)
    torch.cuda.synchronize()
    a.check(ya)
    b.check(yb)


# ------------------------------------------------------ offsets past 32 bits

def test_route_of_many_tokens():
    """More than 2^31 logits: the last tokens as in a batch of their own."""
    n, e, k = (1 << 23) + 777, 260, 6
    l = torch.empty(n, e, dtype=torch.bfloat16, device=G.dev()).normal_()
    ids = torch.full((n, k), -1, dtype=torch.int32, device=G.dev())
    w = torch.zeros(n, k, device=G.dev())
    mb.route(mb.RouteParams.make(n, e, k, dtype="bf16"), l, ids, w)
    tail = l[-500:].clone()
    ids2, w2 = torch.empty_like(ids[:500]), torch.empty_like(w[:500])
    mb.route(mb.RouteParams.make(500, e, k, dtype="bf16"), tail, ids2, w2)
    assert torch.equal(ids[-500:], ids2) and torch.equal(w[-500:], w2)
    want, _ = R.route(f64(tail[-50:]), k)
    assert np.array_equal(ids[-50:].cpu().numpy(), want)


def test_norm_and_4_bit_rows_past_32_bits():
    n, h = 290_003, 7680  # 2.2e9 elements
    x = torch.empty(n, h, dtype=torch.bfloat16, device=G.dev()).normal_()
    w = torch.ones(h, dtype=torch.bfloat16, device=G.dev())
    q = torch.empty(n, h, dtype=torch.uint8, device=G.dev())
    qs = torch.empty(n, h // 128, device=G.dev())
    y = torch.empty_like(x)
    mb.rmsnorm_fp8(x, w, 1e-6, q, qs, residual=x, residual_out=y)
    tail = x[-300:].clone()
    q2, qs2, y2 = torch.empty_like(q[:300]), torch.empty_like(qs[:300]), torch.empty_like(tail)
    mb.rmsnorm_fp8(tail, w, 1e-6, q2, qs2, residual=tail, residual_out=y2)
    assert torch.equal(q[-300:], q2) and torch.equal(qs[-300:], qs2) and torch.equal(y[-300:], y2)
    assert torch.equal(y2, 2 * tail)
    c = q.view(-1)[: n * h // 2].view(n, h // 2)
    s = torch.empty(n, h // 32, dtype=torch.uint8, device=G.dev())
    mb.quantize_mx4(x, c, s)
    mb.dequantize_mx4(c, s, y)
    for at in (0, n // 2, n - 3):
        v = f64(x[at:at + 3])
        ws = R.mx4_scale_bytes(v)
        assert np.array_equal(f64(y[at:at + 3]), R.mx4_values(R.pack4(R.mx4_codes(v, ws)), ws))


@pytest.mark.parametrize("tokens", [64, 1 << 20])
def test_expert_rows_past_32_bits(tokens):
    """Rows and outputs of more than 2^32 bytes, by each way to the product."""
    n, k, cap = 2048, 7168, 1_200_003
    cu = np.array([[0, cap]], np.int32)
    p = Product(1, 1, 1, 0, 4, n, k, tokens=tokens, plan=(cu, np.full((1, 1), -1, np.int32)))
    p.dims = mb.Dims.make(tokens, 1, 1, 1, 0, 128, cap=cap)
    if tokens == 64:  # this many rows in tiles of 16 take long: the last ones alone
        p.bufs.cu_seqlens.copy_(torch.tensor([[cap - 700, cap]], dtype=torch.int32))
    p.bufs.row_src = torch.empty(cap, dtype=torch.int32, device=G.dev())
    p.dev[0] = torch.randint(0, 256, (cap, k // 2), dtype=torch.uint8, device=G.dev())
    p.dev[1] = torch.randint(124, 130, (cap, k // 32), dtype=torch.uint8, device=G.dev())
    y = torch.full((cap, n), -77.0, dtype=torch.bfloat16, device=G.dev())
    p.run(y)
    a = R.mx4_values(p.dev[0][-40:].cpu().numpy(), p.dev[1][-40:].cpu().numpy())
    w = R.mx4_values(p.w, p.w_s)
    want, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    err = np.abs(f64(y[-40:]) - want)
    assert np.all(err <= k * 2.0**-23 * mag + 2.0**-8 * np.abs(want) + 1e-30)
    assert (y[:100] == -77).all() == (tokens == 64)


# -------------------------------------------------------------- a whole layer

def plain_layer(c, ids, w, xr, wg, wd):
    """The layer's output in 64 bits from 4-bit rows (values) and weights,
    re-quantising the intermediate rows as the layer does."""
    y = np.zeros((c["N"], c["H"]))
    for t in range(c["N"]):
        for j in range(c["K"]):
            e = ids[t, j]
            up = R.bf16_round(np.float32(xr[t] @ wg[e].T))[None]
            v = R.swiglu(up)
            s = R.mx4_scale_bytes(v)
            a = R.mx4_values(R.pack4(R.mx4_codes(v, s)), s)
            y[t] += w[t, j] * (a @ wd[e].T)[0]
    return y


class Layer:
    """logits -> route -> plan; x -> norm -> 4-bit rows -> dispatch -> expert
    products with the gated activation between -> combine."""

    def __init__(self, seed=1, N=64, H=256, I=128, E=16, K=4, P=4, R_=1, cap_factor=2):
        self.c = dict(N=N, H=H, I=I, E=E, K=K)
        r = rng(seed)
        g = G.dev()
        self.cap = N // P * K * cap_factor
        self.dims = mb.Dims.make(N, K, E, P, R_, H, cap=self.cap, dtype_in="mx4")
        self.fp8 = mb.Dims.make(N, K, E, P, R_, H, cap=self.cap, dtype_in="fp8")
        self.prm = mb.RouteParams.make(N, E, K, score="sigmoid", n_groups=4, top_groups=2,
                                       group_top=2, scale=2.5)
        self.x = R.bf16_round(np.float32(r.standard_normal((N, H))))
        self.res = R.bf16_round(np.float32(r.standard_normal((N, H))))
        self.gain = R.bf16_round(np.float32(1 + 0.1 * r.standard_normal(H)))
        self.logits = np.float32(r.standard_normal((N, E)))
        self.bias = np.float32(0.05 * r.standard_normal(E))
        rows = P * self.cap
        self.wg, self.wd = (r.integers(0, 256, (E, o, i // 2), dtype=np.uint8)
                            for o, i in ((2 * I, H), (H, I)))
        self.wgs, self.wds = (r.integers(120, 123, (E, o, i // 32), dtype=np.uint8)
                              for o, i in ((2 * I, H), (H, I)))
        e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=g)  # noqa: E731
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=g)  # noqa: E731
        self.t = dict(
            x=dev(self.x, torch.bfloat16), res=dev(self.res, torch.bfloat16),
            gain=dev(self.gain, torch.bfloat16), logits=dev(self.logits), bias=dev(self.bias),
            wg=dev(self.wg), wgs=dev(self.wgs), wd=dev(self.wd), wds=dev(self.wds),
            ids=torch.zeros(N, K, dtype=torch.int32, device=g), w=torch.zeros(N, K, device=g),
            res_out=bf(N, H), normed=bf(N, H), q8=e8(N, H), s8=torch.zeros(N, H // 128, device=g),
            q4=e8(N, H // 2), s4=e8(N, H // 32), buf=e8(rows, H // 2), buf_s=e8(rows, H // 32),
            buf8=e8(rows, H), buf8_s=torch.zeros(rows, H // 128, device=g), up=bf(rows, 2 * I),
            mid=e8(rows, I // 2), mid_s=e8(rows, I // 32), down=bf(rows, H), y=bf(N, H))
        self.bufs = mb.PlanBuffers.allocate(self.dims, g)
        self.ws = mb.alloc_workspace(self.dims, g)

    def run(self):
        t, d, b = self.t, self.dims, self.bufs
        H, I = self.c["H"], self.c["I"]
        mb.rmsnorm_fp8(t["x"], t["gain"], 1e-6, t["q8"], t["s8"], residual=t["res"],
                       residual_out=t["res_out"], y=t["normed"])
        mb.route(self.prm, t["logits"], t["ids"], t["w"], bias=t["bias"])
        mb.plan(d, t["ids"], self.ws, b)
        mb.dispatch(self.fp8, b, t["q8"], t["buf8"], t["s8"], t["buf8_s"])
        mb.quantize_mx4(t["normed"], t["q4"], t["s4"])
        mb.dispatch(d, b, t["q4"], t["buf"], t["s4"], t["buf_s"])
        mb.expert_mx4(d, b, 2 * I, H, t["buf"], t["buf_s"], t["wg"], t["wgs"], t["up"])
        mb.quantize_mx4(t["up"], t["mid"], t["mid_s"], act="swiglu", row_src=b.row_src)
        mb.expert_mx4(d, b, H, I, t["mid"], t["mid_s"], t["wd"], t["wds"], t["down"])
        mb.combine(d, b, t["down"], t["w"], t["y"])

    def check(self):
        torch.cuda.synchronize()
        t, c = self.t, self.c
        ids, w = R.route(self.logits, c["K"], "sigmoid", bias=self.bias, n_groups=4, top_groups=2,
                         group_top=2, scale=2.5)
        assert np.array_equal(t["ids"].cpu().numpy(), ids)
        row_src = self.bufs.row_src.cpu().numpy()
        pos = self.bufs.pos.cpu().numpy()
        assert int(self.bufs.status[0]) & mb.ST_FATAL == 0
        # the dispatched rows are the quantised rows of their tokens, scales included
        used = row_src >= 0
        q4, s4 = t["q4"].cpu().numpy(), t["s4"].cpu().numpy()
        assert np.array_equal(t["buf"].cpu().numpy()[used], q4[row_src[used]])
        assert np.array_equal(t["buf_s"].cpu().numpy()[used], s4[row_src[used]])
        assert np.array_equal(t["buf8"].cpu().numpy()[used], t["q8"].cpu().numpy()[row_src[used]])
        assert np.array_equal(t["buf8_s"].cpu().numpy()[used], t["s8"].cpu().numpy()[row_src[used]])
        assert (pos >= 0).all()
        E, H, I = c["E"], c["H"], c["I"]
        wg = R.mx4_values(self.wg.reshape(-1, H // 2), self.wgs.reshape(-1, H // 32)).reshape(
            E, 2 * I, H)
        wd = R.mx4_values(self.wd.reshape(-1, I // 2), self.wds.reshape(-1, I // 32)).reshape(
            E, H, I)
        want = plain_layer(c, ids, w, R.mx4_values(q4, s4), wg, wd)
        # Rounding to 4 bits inside the layer makes single values jump by a
        # step where the two sides round to different neighbours (the bf16
        # rows before it differ by half a step at times). Such values are
        # few: the whole output agrees to the bf16 roundings of its K terms.
        got = f64(t["y"])
        assert np.linalg.norm(got - want) <= 2.0**-6 * np.linalg.norm(want)
        return got


def test_a_layer_from_logits_to_combined_rows():
    layer = Layer()
    layer.run()
    layer.check()


def test_a_layer_replayed_from_a_graph():
    layer = Layer(seed=2)
    layer.run()
    eager = layer.check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer.run()
    for i in range(3):
        layer.t["y"].zero_()
        layer.t["ids"].fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(f64(layer.t["y"]), eager), i
    # new logits and rows through the same graph
    other = Layer(seed=3)
    for n in ("x", "res", "gain", "logits", "bias", "wg", "wgs", "wd", "wds"):
        layer.t[n].copy_(other.t[n])
    graph.replay()
    torch.cuda.synchronize()
    other.run()
    torch.cuda.synchronize()
    assert torch.equal(layer.t["y"], other.t["y"])
    assert not np.array_equal(f64(other.t["y"]), eager)


def test_routed_workload_feeds_the_plan():
    """A routing of a known workload's size through route and plan: the ids
    are distinct and in range, so the plan has no fatal flag."""
    wl = W.get_workload("decode_drift")
    prm = mb.RouteParams.make(wl.n_tokens, wl.n_experts, wl.top_k, score="softmax", dtype="bf16")
    l = torch.randn(wl.n_tokens, wl.n_experts, device=G.dev()).bfloat16()
    dims = mb.Dims.for_workload(wl, cap=4 * wl.cap)
    ids = torch.empty(wl.n_tokens, wl.top_k, dtype=torch.int32, device=G.dev())
    w = torch.empty(wl.n_tokens, wl.top_k, device=G.dev())
    mb.route(prm, l, ids, w)
    bufs = mb.PlanBuffers.allocate(dims, G.dev())
    mb.plan(dims, ids, mb.alloc_workspace(dims, G.dev()), bufs)
    assert mb.plan_status(bufs)[0] & mb.ST_FATAL == 0
    assert torch.allclose(w.sum(1), torch.ones(wl.n_tokens, device=G.dev()), atol=1e-5)
