"""Corners of the router, the norm, the 4-bit rows and their dispatch on the
GPU, each against its plain definition."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import token_dispatch_mb_amd as mb

from . import gpu_harness as G
from . import plain_ops as R
from .test_gpu_ops import Product, check_norm, dev, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_required():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


# -------------------------------------------------------------------- norm

@pytest.mark.parametrize("n,h", [(1, 128), (513, 384), (200, 7168)])
def test_norm_codes_are_the_quotients(n, h):
    """scale = max|y| / 448 and q = e4m3fn(y / scale), both as binary32
    division rounds them: from the normed rows that the call returns, exact."""
    r = rng(n, h, 7)
    # short fractions, whose quotients often are midpoints of two codes
    x = np.round(r.standard_normal((n, h)) * 16) / 16
    x[:, ::128] = 4.0
    x = dev(np.float32(x * np.exp2(r.integers(-20, 20, (n, 1)))))
    w = dev(np.float32(1 + np.round(r.standard_normal(h)) / 16))
    q = torch.full((n, h), 0xA5, dtype=torch.uint8, device=G.dev())
    qs = torch.full((n, h // 128), -5.0, device=G.dev())
    y = torch.empty_like(x)
    mb.rmsnorm_fp8(x, w, 0.0, q, qs, y=y)
    yy = y.cpu().numpy().reshape(n, h // 128, 128)
    scale = np.abs(yy).max(axis=2) / np.float32(448)
    assert scale.dtype == np.float32
    assert np.array_equal(qs.cpu().numpy(), scale)
    want = torch.from_numpy((yy / scale[:, :, None]).reshape(n, h)).to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu(), want.view(torch.uint8))


# ------------------------------------------------------------------- route

def plain_choice(l, k, groups, top_groups, score, bias):
    """The ids of all rows at once in 64 bits, group scores of two experts."""
    l = l.astype(np.float64)
    n, e = l.shape
    if score == "sigmoid":
        c = 1 / (1 + np.exp(-l))
    else:
        c = np.exp(l - l.max(axis=1, keepdims=True))
        c /= c.sum(axis=1, keepdims=True)
    c = c + bias.astype(np.float64)
    g = np.sort(c.reshape(n, groups, -1), axis=2)[:, :, -2:].sum(axis=2)
    first = np.argsort(-g, axis=1, kind="stable")[:, :top_groups]
    closed = np.ones((n, groups), bool)
    np.put_along_axis(closed, first, False, axis=1)
    c[np.repeat(closed, e // groups, axis=1)] = -np.inf
    return np.argsort(-c, axis=1, kind="stable")[:, :k]


@pytest.mark.parametrize("e,k", [(64, 6), (256, 8)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("at", [-1.0, -8.0, -12.0, -25.0, -44.0, -60.0, -68.0, -80.0])
def test_route_far_logits_in_groups(at, score, e, k):
    """Scores far below one, close together: their binary32 values are off by
    their logit's size, and what that leaves open is decided in binary64."""
    n = 20000
    r = rng(e, int(-at), len(score))
    l = np.float32(at + 0.01 * r.uniform(-1, 1, (n, e)))
    if score == "softmax":
        l[:, 0] = 0.0
    elif at == -44.0:  # two groups' sums, 8.532099599e-20 and 8.532099253e-20
        s = e // 8
        l[0] = -90.0
        l[0, 0], l[0, 1] = -44.579517, -44.622982
        l[0, s], l[0, s + 1] = -44.590237, -44.611908
        l[0, 2 * s::s] = -40.0
        l[0, 5 * s::s] = -90.0  # those two groups fight for the last open place
    disabled = np.zeros(e, np.float32)
    disabled[e - 1] = -1e9
    prm = mb.RouteParams.make(n, e, k, score=score, n_groups=8, top_groups=4, group_top=2)
    ids = torch.empty(n, k, dtype=torch.int32, device=G.dev())
    w = torch.empty(n, k, device=G.dev())
    x = dev(l)
    for bias in (None, np.zeros(e, np.float32), disabled):
        want = plain_choice(l, k, 8, 4, score, np.zeros(e) if bias is None else bias)
        mb.route(prm, x, ids, w, bias=None if bias is None else dev(bias))
        wrong = np.nonzero((ids.cpu().numpy() != want).any(axis=1))[0]
        assert not len(wrong), (len(wrong), wrong[:5], ids[wrong[0]], want[wrong[0]])


# ---------------------------------------------------------------- overlaps

def test_outputs_beside_their_inputs_and_over_them():
    """Buffers that touch in one allocation are separate ones; outputs over
    inputs are refused with the reason."""
    g = G.dev()
    mem = torch.zeros(1 << 16, dtype=torch.uint8, device=g)

    def part(lo, n, dtype, *shape):
        return mem[lo:lo + n].view(dtype).view(*shape)

    x = torch.randn(4, 256, device=g)
    part(0, 4096, torch.float32, 4, 256).copy_(x)
    q, s = part(4096, 512, torch.uint8, 4, 128), part(4608, 32, torch.uint8, 4, 8)
    mb.quantize_mx4(part(0, 4096, torch.float32, 4, 256), q, s)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    mb.quantize_mx4(x, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    back = part(4640, 2048, torch.bfloat16, 4, 256)
    mb.dequantize_mx4(q, s, back)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    with pytest.raises(ValueError, match="overlap"):
        mb.quantize_mx4(part(0, 4096, torch.float32, 4, 256), part(4080, 512, torch.uint8, 4, 128),
                        s)
    with pytest.raises(ValueError, match="overlap"):
        mb.dequantize_mx4(q, s, part(4624, 2048, torch.bfloat16, 4, 256))

    prm = mb.RouteParams.make(16, 64, 4)
    l = part(0, 4096, torch.float32, 16, 64)
    l.normal_()
    ids, w = part(4096, 256, torch.int32, 16, 4), part(4352, 256, torch.float32, 16, 4)
    mb.route(prm, l, ids, w)
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    mb.route(prm, l, ids2, w2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    with pytest.raises(ValueError, match="overlap"):
        mb.route(prm, l, part(4092, 256, torch.int32, 16, 4), w)

    p = Product(21, 2, 2, 1, 20, 64, 128)
    over = p.dev[2].view(-1)[:p.dims.rows * 64 * 2].view(torch.bfloat16).view(-1, 64)
    with pytest.raises(ValueError, match="overlap"):
        p.run(over)
    p.check(p.run())


# -------------------------------------------------------------- 4-bit rows

@pytest.mark.parametrize("up", [1.0, 3e30])
@pytest.mark.parametrize("lo,hi", [(-100.0, -88.7), (-88.7, -87.3), (-87.3, -80.0), (-30.0, -10.0), (10.0, 90.0)])
def test_swiglu_blocks_of_far_gates(lo, hi, up):
    """Whole blocks whose sigmoids are near or below the smallest normal
    number. The activation in binary32, in units of 2^-24: two exponentials (2
    each) and their corrections (1 each), a sum (1), a reciprocal (2) and four
    products (1 each): 13, below 2^-20 relative, which moves a code only where
    the value is that close to a midpoint."""
    r = rng(abs(int(lo)), 3)
    m, h = 33, 256
    x = np.empty((m, 2 * h), np.float32)
    x[:, :h] = r.uniform(lo, hi, (m, h))
    x[:, h:] = up * r.uniform(0.5, 1.0, (m, h))
    v = R.swiglu(x)
    q = torch.full((m, h // 2), 0xA5, dtype=torch.uint8, device=G.dev())
    s = torch.full((m, h // 32), 0xA5, dtype=torch.uint8, device=G.dev())
    mb.quantize_mx4(dev(x), q, s, act="swiglu")
    s = s.cpu().numpy()
    near = R.mx4_scale_bytes(v * (1 - 2.0**-20)), R.mx4_scale_bytes(v * (1 + 2.0**-20))
    assert ((s == near[0]) | (s == near[1])).all()
    unit = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, axis=1)
    a = np.abs(v) / unit
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0)) * unit
    err = np.abs(R.mx4_values(q.cpu().numpy(), s) - np.clip(v, -6 * unit, 6 * unit))
    assert np.all(err <= half + 2.0**-20 * np.abs(v)), (err / (half + 2.0**-20 * np.abs(v))).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-30, 1e-20])
def test_norm_of_rows_whose_squares_vanish(eps, dtype):
    """Rows down to the smallest numbers: beside an epsilon as small, their
    mean square is what counts, though binary32 does not hold it."""
    r = rng(11)
    x = r.standard_normal((12, 896)) * 10.0 ** -np.arange(14, 50, 3)[:, None]
    x[3, 128:] = 0
    w = 1 + 0.1 * r.standard_normal(896)
    eps = float(np.float32(eps))  # as the call takes it: 1e-42 has 10 bits there
    check_norm(x, w, eps, dtype)
    check_norm(x, w, eps, dtype, residual=0.5 * x[::-1])


def test_norm_of_more_rows_than_one_launch_holds():
    """512 threads to a row, and fewer than 2^32 to a launch: from 2^23 - 2
    rows on there are several, each with its own part of every tensor."""
    n, h = (1 << 23) + 1001, 128
    g = G.dev()
    x = torch.empty(n, h, dtype=torch.bfloat16, device=g).normal_()
    res = torch.empty_like(x).normal_()
    w = torch.empty(h, dtype=torch.bfloat16, device=g).uniform_(0.5, 2)
    q = torch.full((n, h), 0xA5, dtype=torch.uint8, device=g)
    qs = torch.full((n, 1), -5.0, device=g)
    y, out = torch.zeros_like(x), torch.zeros_like(x)
    mb.rmsnorm_fp8(x, w, 1e-6, q, qs, residual=res, residual_out=out, y=y)
    for at in (slice(0, 700), slice((1 << 23) - 400, (1 << 23) + 300), slice(n - 700, n)):
        one = [t[at].clone() for t in (x, res)]
        q1, qs1, y1, o1 = (torch.empty_like(t[at]) for t in (q, qs, y, out))
        mb.rmsnorm_fp8(one[0], w, 1e-6, q1, qs1, residual=one[1], residual_out=o1, y=y1)
        for a, b in ((q, q1), (qs, qs1), (y, y1), (out, o1)):
            assert torch.equal(a[at], b)


# ------------------------------------------------- the dispatch of 4-bit rows

@pytest.mark.parametrize("shift", [0, 4])
@pytest.mark.parametrize("h,k", [(128, 2), (896, 3), (4096, 1), (4096, 2), (4096, 16), (4096, 17),
                                 (7168, 8), (7168, 4), (8192, 8), (8192, 5)])
def test_dispatch_of_4_bit_rows(h, k, shift):
    """Rows of any length, those of whole 2 KiB spans among them, with their
    scales at 16-byte and at other addresses: every row and scale row of the
    plan is its token's, the padding stays as it was."""
    n, e, p = 136, 32, 4
    r = rng(h, k)
    ids = np.stack([r.permutation(e)[:k] for _ in range(n)]).astype(np.int32)
    dims = mb.Dims.make(n, k, e, p, 2, h, cap=2 * n // p * k + 64, dtype_in="mx4")
    plan = G.GpuPlan(dims)
    plan.run(ids)
    x = dev(r.integers(0, 256, (n, h // 2), dtype=np.uint8))
    words = h // 32

    def at(t):  # the same bytes, `shift` behind a 16-byte address
        m = torch.full((t.numel() + shift,), 0xA5, dtype=torch.uint8, device=G.dev())
        m[shift:] = t.reshape(-1)
        return m[shift:].view(t.shape)

    xs = at(dev(r.integers(0, 256, (n, words), dtype=np.uint8)))
    buf = torch.full((dims.rows, h // 2), 0x5A, dtype=torch.uint8, device=G.dev())
    bs = at(torch.full((dims.rows, words), 0x5A, dtype=torch.uint8, device=G.dev()))
    mb.dispatch(dims, plan.bufs, x, buf, xs, bs)
    torch.cuda.synchronize()
    assert int(plan.bufs.status[0]) & mb.ST_FATAL == 0
    src = plan.bufs.row_src.long().view(-1)
    used = src >= 0
    token = src[used]
    assert len(token) == n * k
    assert torch.equal(buf[used], x[token]) and torch.equal(bs[used], xs[token])
    assert (buf[~used] == 0x5A).all() and (bs[~used] == 0x5A).all()
