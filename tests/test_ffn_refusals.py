"""The experts' products from bf16 rows, their gradients, the combine's
gradients and the projection with adapters refuse, on the host and before
anything is launched, what the header does not allow; the binding refuses
tensors the kernels cannot take. Their definitions are pinned by hand and by
differences. All of it runs without a GPU."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import token_dispatch_mb_amd as mb

from . import plain_ffn as F

vp = ctypes.c_void_p
BAD, WS = mb.ERR_INVALID_ARG, mb.ERR_WORKSPACE
MB = 1 << 20


def at(i, off=0):
    """An address 64 MB from the others (never dereferenced)."""
    return vp(64 * MB * (i + 1) + off)


def _dims(**kw):
    return mb.Dims.make(**{**dict(n_tokens=64, top_k=2, n_experts=16, n_ranks=4, slots_per_rank=1,
                                  hidden=128), **kw})


def _bufs(**kw):
    return mb._PlanBufsC(**{n: kw.get(n, 1 << 20) for n, _ in mb._PlanBufsC._fields_})


def _product(d=None, bufs=None, act=0, n=64, k=128, a=at(0), w=at(1), y=at(2), pre=None):
    d, bufs = d or _dims(), bufs or _bufs()
    return mb.raw_call("mb_expert_bf16", ctypes.byref(d), ctypes.byref(bufs), act, n, k, a, w, y, pre,
                       None)


def _dgrad(d=None, bufs=None, act=0, n=64, k=128, a=at(0), w=at(1), y=at(2), pre=None):
    d, bufs = d or _dims(), bufs or _bufs()
    return mb.raw_call("mb_expert_bf16_dgrad", ctypes.byref(d), ctypes.byref(bufs), act, n, k, a, w,
                       pre, y, None)


def _wgrad(d=None, bufs=None, act=0, n=64, k=128, a=at(0), w=at(1), y=at(2), pre=None, add=0):
    """act: the type of dw."""
    d, bufs = d or _dims(), bufs or _bufs()
    return mb.raw_call("mb_expert_bf16_wgrad", ctypes.byref(d), ctypes.byref(bufs), n, k, act, add, a,
                       w, y, None)


CALLS = [_product, _dgrad, _wgrad]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=-8), dict(n=12), dict(n=4), dict(n=MB + 8), dict(k=0), dict(k=-8), dict(k=20),
    dict(k=MB + 8), dict(act=2), dict(act=-1), dict(a=None), dict(w=None), dict(y=None),
    dict(a=at(0, 8)), dict(w=at(1, 8)), dict(y=at(2, 8)), dict(d=_dims(n_tokens=63)),
    dict(d=_dims(dtype_out="fp8")), dict(bufs=_bufs(status=None)), dict(bufs=_bufs(cu_seqlens=None)),
    dict(bufs=_bufs(rep_expert=None)), dict(d=_dims(cap=1 << 28), n=MB), dict(d=_dims(cap=1 << 28), k=MB),
    dict(d=_dims(n_tokens=4, n_ranks=1, cap=(1 << 31) - 256)),
    dict(d=_dims(n_experts=1024, n_ranks=1), n=MB, k=MB), dict(y=at(0)), dict(y=at(1)),
    dict(y=at(0, 16)), dict(y=vp(1 << 20)),
])
def test_products_refuse(call, kw):
    assert call(**kw) == BAD


@pytest.mark.parametrize("call", [_product, _dgrad])
def test_products_need_pre_with_the_activation_only(call):
    assert call(pre=at(3)) == BAD
    assert call(act=1, pre=at(3, 8)) == BAD
    for over in (at(0), at(1), at(2), vp(1 << 20)):
        if call is _product or over.value == at(2).value:
            assert call(act=1, pre=over) == BAD
    if call is _dgrad:
        assert call(act=1) == BAD


def test_a_wider_weight_and_output_with_the_activation():
    # w is [E, 2n, k]: 16 * 64 * 2 * 128 * 2 bytes; y one byte behind its first half overlaps it
    w = 64 * MB * 2
    assert _product(act=1, y=vp(w + 16 * 64 * 128 * 2)) == BAD
    # da is [rows, 2k]
    rows = _dims().rows
    assert _dgrad(act=1, pre=at(3), a=vp(64 * MB * 3 + rows * 128 * 2)) == BAD


@pytest.mark.parametrize("call", [_product, _dgrad])
def test_products_without_tokens_do_nothing(call):
    assert call(d=_dims(n_tokens=0)) == mb.OK


def _comb(d=None, bufs=None, dy=at(0), ye=at(1), w=at(2), dye=at(3), dw=at(4)):
    d, bufs = d or _dims(), bufs or _bufs()
    return mb.raw_call("mb_combine_grad", ctypes.byref(d), ctypes.byref(bufs), dy, ye, w, dye, dw,
                       None)


@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(ye=None), dict(w=None), dict(dye=None, dw=None), dict(dy=at(0, 8)),
    dict(ye=at(1, 8)), dict(w=at(2, 2)), dict(dye=at(3, 8)), dict(dw=at(4, 2)),
    dict(bufs=_bufs(status=None)), dict(bufs=_bufs(pos=None)), dict(d=_dims(n_tokens=63)),
    dict(dye=at(0)), dict(dye=at(1)), dict(dye=at(2)), dict(dw=at(0)), dict(dw=at(1, 16)),
    dict(dw=at(2)), dict(dw=at(3)), dict(dw=vp(1 << 20)), dict(dye=vp(1 << 20)),
])
def test_combine_grad_refuses(kw):
    assert _comb(**kw) == BAD


def test_combine_grad_without_tokens_does_nothing():
    assert _comb(d=_dims(n_tokens=0), dy=None, ye=None, w=None) == mb.OK


def _lora(prm=None, x=at(0), w=at(1), a=at(2), b=at(3), scale=at(4), ad=at(5), ws=at(6),
          nbytes=64 * MB, y=at(7), **kw):
    prm = prm or mb.LoraParams.make(**{**dict(n_rows=20, n_out=64, k_in=128, rank=16, n_adapters=3),
                                       **kw})
    return mb.raw_call("mb_project_lora", ctypes.byref(prm), x, w, a, b, scale, ad, ws, nbytes, y, None)


SIZES = [dict(n_rows=-1), dict(n_rows=(1 << 26) + 1), dict(n_out=0), dict(n_out=12), dict(n_out=-8),
         dict(n_out=MB + 8), dict(k_in=0), dict(k_in=12), dict(k_in=MB + 8), dict(rank=0),
         dict(rank=12), dict(rank=-8), dict(rank=264), dict(n_adapters=0), dict(n_adapters=MB + 1),
         dict(dtype_out="fp8"), dict(dtype_out=-1), dict(n_rows=1 << 26, n_out=MB)]


@pytest.mark.parametrize("kw", SIZES)
def test_lora_refuses_sizes(kw):
    assert _lora(**kw) == BAD
    prm = mb.LoraParams.make(**{**dict(n_rows=20, n_out=64, k_in=128, rank=16, n_adapters=3), **kw})
    assert mb.lora_workspace_bytes(prm) == 0
    with pytest.raises(mb.MoebalError):
        mb.alloc_lora_workspace(prm, "cpu")


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(a=None), dict(b=None), dict(scale=None), dict(ad=None),
    dict(ws=None), dict(y=None), dict(x=at(0, 8)), dict(w=at(1, 8)), dict(a=at(2, 8)),
    dict(b=at(3, 8)), dict(scale=at(4, 2)), dict(ad=at(5, 2)), dict(ws=at(6, 8)), dict(y=at(7, 8)),
    dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(y=at(4)), dict(y=at(5)),
    dict(y=at(6)), dict(ws=at(0)), dict(ws=at(1)), dict(ws=at(5)),
])
def test_lora_refuses_pointers(kw):
    assert _lora(**kw) == BAD


def test_lora_workspace():
    prm = mb.LoraParams.make(20, 64, 128, 16, 3)
    need = mb.lora_workspace_bytes(prm)
    assert need >= 20 * 16 * 4
    assert _lora(prm, nbytes=need - 1) == WS
    assert mb.raw_call("mb_project_lora", None, *([at(0)] * 7), 64 * MB, at(7), None) == BAD
    assert mb.lora_workspace_bytes(mb.LoraParams.make(0, 64, 128, 16, 3)) > 0
    assert _lora(n_rows=0, x=None, w=None, a=None, b=None, scale=None, ad=None, ws=None, nbytes=0,
                 y=None) == mb.OK


def test_binding_refuses_host_tensors():
    z = torch.zeros
    h = z(4096, dtype=torch.bfloat16)
    d = _dims()
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.expert_bf16(d, None, 64, 128, h, h, h)
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.expert_bf16_dgrad(d, None, 64, 128, h, h, h)
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.expert_bf16_wgrad(d, None, 64, 128, h, h, z(64))
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.combine_grad(d, None, h, h, z(64), h)
    with pytest.raises(ValueError, match="GPU tensor"):
        mb.project_lora(mb.LoraParams.make(4, 64, 128, 16, 3), h, h, h, h, z(3), z(4), z(9), h)
    with pytest.raises(KeyError):
        mb.expert_bf16(d, None, 64, 128, h, h, h, act="relu")


# ------------------------------------------ the definitions pinned

def test_definition_of_the_gated_product_by_hand():
    a = np.array([[1.0, 2.0]])
    w = np.array([[1.0, 1.0], [0.0, 0.0], [2.0, 0.0], [0.0, -1.0]])  # two gates, two ups
    g, _, u, _, h, _ = F.gated(a, w)
    assert g.tolist() == [[3, 0]] and u.tolist() == [[2, -2]]
    assert np.allclose(h, [[3 / (1 + np.exp(-3)) * 2, 0]])
    # far gates keep their value: silu(-88) = -88 exp(-88) to 38 digits
    assert np.isclose(F.sigmoid(np.array(-88.0)) / np.exp(-88.0), 1)


def test_gradients_of_the_block_by_differences():
    """The gradients that the definitions give for sum(dy * block(x)), against
    central differences in every weight and input."""
    r = np.random.default_rng(3)
    m, h, i = 3, 4, 2
    x, w1, w2 = r.standard_normal((m, h)), r.standard_normal((2 * i, h)), r.standard_normal((h, i))
    dy = r.standard_normal((m, h))

    def value():
        return float((F.gated(x, w1)[4] @ w2.T * dy).sum())

    g, _, u, _, mid, _ = F.gated(x, w1)
    dg, _, du, _ = F.gate_grad(dy, w2, g, u)
    dpre = np.concatenate((dg, du), axis=1)
    grads = [(x, F.row_grad(dpre, w1)[0]), (w1, F.weight_grad(dpre, x)[0]),
             (w2, F.weight_grad(dy, mid)[0])]
    for t, want in grads:
        for j in np.ndindex(t.shape):
            keep, e = t[j], 1e-5
            t[j] = keep + e
            up = value()
            t[j] = keep - e
            down = value()
            t[j] = keep
            assert abs((up - down) / (2 * e) - want[j]) < 1e-8 * max(1, abs(want[j])) + 1e-8


def test_gradients_of_the_combine_by_differences():
    r = np.random.default_rng(4)
    pos = np.array([[0, 3], [2, 1]])
    w, y, dy = r.standard_normal((2, 2)), r.standard_normal((4, 5)), r.standard_normal((2, 5))
    rows, dw, _ = F.combine_grad(pos, w, dy, y)
    e = 1e-6
    for j in np.ndindex(w.shape):
        v = w.copy()
        v[j] += e
        got = ((F.combine(pos, v, y) - F.combine(pos, w, y)) * dy).sum() / e
        assert abs(got - dw[j]) < 1e-6
    for t, k in np.ndindex(pos.shape):
        for i in range(5):
            v = y.copy()
            v[pos[t, k], i] += e
            got = ((F.combine(pos, w, v) - F.combine(pos, w, y)) * dy).sum() / e
            assert abs(got - rows[t, k, i]) < 1e-6


def test_definition_of_the_adapters_by_hand():
    x, w = np.array([[1.0, 2.0], [1.0, 2.0]]), np.array([[1.0, 0.0]])
    a, b = np.array([[[0.0, 1.0]]]), np.array([[[10.0]]])
    y, _ = F.lora(x, w, a, b, np.array([0.5]), [0, -1])
    assert y.tolist() == [[11.0], [1.0]]  # 1 + 10 * (0.5 * 2), and without
