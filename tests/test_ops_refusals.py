"""The router, the norm, the 4-bit rows and the experts' products refuse, on
the host and before anything is launched, sizes, types, alignments and null
pointers outside what the header allows; the binding refuses tensors the
kernels cannot take. All of it runs without a GPU."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import token_dispatch_mb_amd as mb

from . import plain_ops as R

vp = ctypes.c_void_p
A = vp(1 << 20)  # aligned, never dereferenced
ODD = vp((1 << 20) + 2)
EIGHT = vp((1 << 20) + 8)
BAD = mb.ERR_INVALID_ARG


def _route(prm, logits=A, bias=None, ids=A, w=A):
    return mb.raw_call("mb_route", ctypes.byref(prm), logits, bias, ids, w, None)


@pytest.mark.parametrize("kw", [
    dict(n_tokens=-1), dict(n_tokens=1 << 26), dict(n_experts=0), dict(n_experts=1025),
    dict(top_k=0), dict(top_k=33), dict(n_experts=8, top_k=9), dict(dtype=2), dict(dtype=3),
    dict(dtype=-1), dict(score=2), dict(score=-1), dict(n_groups=0), dict(n_groups=3),
    dict(n_experts=1024, n_groups=128, top_groups=64), dict(n_groups=8, top_groups=0),
    dict(n_groups=8, top_groups=9), dict(group_top=0), dict(group_top=3),
    dict(n_experts=8, n_groups=8, top_groups=8, group_top=2),
    dict(n_experts=32, n_groups=8, top_groups=1, top_k=5),
    dict(scale=float("nan")), dict(scale=float("inf")),
])
def test_route_refuses_parameters(kw):
    base = dict(n_tokens=16, n_experts=64, top_k=4)
    p = mb.RouteParams.make(**{**base, **kw})
    assert _route(p) == BAD


def test_route_refuses_pointers():
    p = mb.RouteParams.make(16, 64, 4)
    assert mb.raw_call("mb_route", None, A, None, A, A, None) == BAD
    for kw in (dict(logits=None), dict(ids=None), dict(w=None), dict(logits=EIGHT),
               dict(bias=ODD), dict(ids=ODD), dict(w=ODD)):
        assert _route(p, **kw) == BAD, kw
    assert _route(mb.RouteParams.make(0, 64, 4), logits=None, ids=None, w=None) == mb.OK


def _norm(n=4, h=128, dtype=mb.BF16, eps=1e-6, x=A, res=None, weight=A, res_out=None, y=None, q=A,
          qs=A):
    return mb.raw_call("mb_rmsnorm_fp8", n, h, dtype, eps, x, res, weight, res_out, y, q, qs, None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=1 << 24), dict(h=0), dict(h=64), dict(h=130), dict(h=16384 + 128),
    dict(dtype=mb.FP8_E4M3), dict(dtype=7), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(x=None), dict(weight=None), dict(q=None), dict(qs=None),
    dict(res_out=A), dict(x=EIGHT), dict(res=EIGHT), dict(weight=EIGHT), dict(res=A, res_out=EIGHT),
    dict(y=EIGHT), dict(q=EIGHT), dict(qs=ODD),
])
def test_norm_refusals(kw):
    assert _norm(**kw) == BAD


def test_norm_of_no_rows():
    assert _norm(n=0, x=None, weight=None, q=None, qs=None) == mb.OK


def _quant(m=4, h=32, dtype=mb.BF16, act=mb.ACT_NONE, x=A, src=None, q=A, qs=A):
    return mb.raw_call("mb_quantize_mx4", m, h, dtype, act, x, src, q, qs, None)


def _dequant(m=4, h=32, dtype=mb.BF16, q=A, qs=A, x=A):
    return mb.raw_call("mb_dequantize_mx4", m, h, dtype, q, qs, x, None)


@pytest.mark.parametrize("kw", [
    dict(m=-1), dict(h=0), dict(h=16), dict(h=48), dict(h=-32), dict(dtype=mb.FP8_E4M3),
    dict(dtype=mb.MX4), dict(m=1 << 26), dict(m=1 << 20, h=1 << 16), dict(x=None), dict(q=None),
    dict(qs=None), dict(x=EIGHT), dict(q=EIGHT),
])
def test_quantize_and_dequantize_refusals(kw):
    assert _quant(**kw) == BAD
    assert _dequant(**kw) == BAD


def test_quantize_refusals():
    assert _quant(act=2) == BAD
    assert _quant(act=-1) == BAD
    assert _quant(src=ODD) == BAD
    assert _quant(m=0, x=None, q=None, qs=None) == mb.OK
    assert _dequant(m=0, x=None, q=None, qs=None) == mb.OK


def _dims(**kw):
    return mb.Dims.make(**{**dict(n_tokens=64, top_k=2, n_experts=16, n_ranks=4, slots_per_rank=1,
                                  hidden=128), **kw})


def _bufs(**kw):
    return mb._PlanBufsC(**{n: kw.get(n, 1 << 20) for n, _ in mb._PlanBufsC._fields_})


def _expert(d=None, bufs=None, n=64, k=128, a=A, a_s=A, w=A, w_s=A, y=A):
    d = d or _dims()
    bufs = bufs or _bufs()
    return mb.raw_call("mb_expert_mx4", ctypes.byref(d), ctypes.byref(bufs), n, k, a, a_s, w, w_s, y,
                       None)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=-8), dict(n=12), dict(n=(1 << 20) + 8), dict(k=0), dict(k=64), dict(k=160),
    dict(k=(1 << 20) + 128), dict(a=None), dict(a_s=None), dict(w=None), dict(w_s=None),
    dict(y=None), dict(a=EIGHT), dict(w=EIGHT), dict(y=EIGHT), dict(a_s=ODD), dict(w_s=ODD),
    dict(d=_dims(n_tokens=63)), dict(d=_dims(dtype_out="fp8")), dict(bufs=_bufs(status=None)),
    dict(bufs=_bufs(cu_seqlens=None)), dict(bufs=_bufs(rep_expert=None)),
    dict(d=_dims(cap=1 << 28), n=1 << 20),
])
def test_expert_refusals(kw):
    assert _expert(**kw) == BAD


def test_expert_without_tokens_does_nothing():
    assert _expert(d=_dims(n_tokens=0)) == mb.OK


def test_mx4_rows_in_the_dispatch_need_whole_words():
    d = _dims(dtype_in="mx4", hidden=128)
    assert mb.workspace_bytes(d) > 0
    assert mb.workspace_bytes(_dims(dtype_in="mx4", hidden=64)) == 0
    b = _bufs()

    def call(x=A, xs=A, buf=A, bs=A):
        return mb.raw_call("mb_dispatch", ctypes.byref(d), ctypes.byref(b), x, xs, buf, bs, None)

    for kw in (dict(xs=None), dict(bs=None), dict(xs=ODD), dict(bs=ODD), dict(x=EIGHT)):
        assert call(**kw) == BAD, kw
    # the combine's rows are never 4-bit ones
    assert mb.workspace_bytes(_dims(dtype_out="mx4")) == 0


def test_binding_refuses_host_tensors():
    z = torch.zeros
    p = mb.RouteParams.make(4, 8, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.route(p, z(4, 8), z(4, 2, dtype=torch.int32), z(4, 2))
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.rmsnorm_fp8(z(4, 128), z(128), 1e-6, z(4, 128, dtype=torch.uint8), z(4, 1))
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.quantize_mx4(z(4, 32), z(4, 16, dtype=torch.uint8), z(4, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.dequantize_mx4(z(4, 16, dtype=torch.uint8), z(4, 1, dtype=torch.uint8), z(4, 32))
    with pytest.raises(ValueError, match="GPU tensor"):
        u = z(4096, dtype=torch.uint8)
        mb.expert_mx4(_dims(), None, 64, 128, u, u, u, u, z(64))
    with pytest.raises(KeyError):
        mb.RouteParams.make(4, 8, 2, score="linear")


# ------------------------------------------ the definitions pinned by hand

def test_definition_of_the_route_by_hand():
    # sigmoid of 0 is 1/2; the bias moves the choice, not the weight
    ids, w = R.route([[0.0, 0.0, 0.0, 0.0]], 2, "sigmoid", bias=[0, 0.1, 0, 0.2], renorm=False)
    assert ids.tolist() == [[3, 1]] and w.tolist() == [[0.5, 0.5]]
    # ties go to the lowest id; weights share the sum
    ids, w = R.route([[1.0, 1.0, 1.0]], 2, "softmax", scale=3.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 1.5)
    # two groups: the best single expert sits in the group of lower pair sum
    l = [[3.0, -9.0, 2.0, 2.0]]
    assert R.route(l, 1, "sigmoid", n_groups=2, top_groups=1, group_top=1)[0].tolist() == [[0]]
    assert R.route(l, 1, "sigmoid", n_groups=2, top_groups=1, group_top=2)[0].tolist() == [[2]]
    # masks: all of a row, and all but one expert
    ids, w = R.route([[-np.inf] * 3, [np.nan, 5.0, -np.inf]], 2, "softmax")
    assert ids.tolist() == [[0, 1], [1, 0]] and w.tolist() == [[0, 0], [1, 0]]


def test_definition_of_the_rows_by_hand():
    v = np.zeros((1, 32))
    v[0, :8] = [7.9, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0]  # ties go to even codes
    s = R.mx4_scale_bytes(v)
    assert s.tolist() == [[127]]
    assert R.mx4_codes(v, s)[0, :8].tolist() == [7, 0, 2, 2, 4, 4, 6, 8 + 6]
    q = R.pack4(R.mx4_codes(v, s))
    assert q[0, 0] == 7 and q[0, 1] == 2 + 2 * 16
    assert R.mx4_values(q, s)[0, :8].tolist() == [6, 0, 1, 1, 2, 2, 4, -4]
    assert R.mx4_scale_bytes(np.full((1, 32), 2.0**-140)).tolist() == [[0]]
    assert R.mx4_scale_bytes(np.full((1, 32), np.nan)).tolist() == [[255]]
    # e4m3: the largest value, the smallest normal and subnormal, NaN
    assert R.e4m3_values(np.array([0x7E, 0x08, 0x01])).tolist() == [448, 2.0**-6, 2.0**-9]
    assert np.isnan(R.e4m3_values(np.array([0x7F]))).all()


def test_definition_of_the_norm_by_hand():
    x = np.zeros((2, 128))
    x[0, 0], x[0, 1] = 3.0, 4.0  # mean square 25 / 128
    h, y, scale = R.rmsnorm(x, np.ones(128), 0.0)
    assert np.allclose(y[0, :2], np.array([3.0, 4.0]) / np.sqrt(25 / 128))
    assert np.allclose(scale[0], y[0, 1] / 448) and scale[1] == 1 and not y[1].any()
    assert np.array_equal(h, x)
