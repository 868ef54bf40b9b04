"""What the router, the norm, the 4-bit rows and the experts' products refuse
beyond single arguments' ranges. All of it runs without a GPU: no call here
gets as far as a launch."""
from __future__ import annotations

import ctypes

import pytest

import token_dispatch_mb_amd as mb

from .test_ops_refusals import A, BAD, _bufs, _dims


def _expert_of_no_tokens(**kw):
    """mb_expert_mx4 without tokens: its checks, and nothing to launch."""
    d, b = _dims(n_tokens=0, **kw), _bufs()
    return mb.raw_call("mb_expert_mx4", ctypes.byref(d), ctypes.byref(b), 8, 128, A, A, A, A,
                       ctypes.c_void_p(1 << 40), None)


@pytest.mark.parametrize("ranks", [1, 3])
def test_expert_rows_are_numbered_up_to_a_tile_behind_the_last(ranks):
    """A tile that ends in the buffer's last rows numbers up to 255 behind
    them: 2^31 - 1 holds those of P*cap = 2^31 - 256, and no more."""
    cap = (2**31 - 256) // ranks
    experts = dict(n_experts=4 * ranks, n_ranks=ranks)
    assert _expert_of_no_tokens(cap=cap, **experts) == mb.OK
    assert _expert_of_no_tokens(cap=cap + 1, **experts) == BAD
    assert _expert_of_no_tokens(cap=(2**31 - 1) // ranks, **experts) == BAD


# A call outside these tests' bounds would be launched, so they are all calls
# that must be refused: addresses whose ranges overlap by one unit at least.
P = ctypes.c_void_p
B0 = 1 << 20  # where the first buffer of each call lies


def _route(logits, bias, ids, w):
    p = mb.RouteParams.make(16, 64, 4)  # logits 4096 bytes, bias 256, ids and w 256 each
    return mb.raw_call("mb_route", ctypes.byref(p), P(logits), P(bias), P(ids), P(w), None)


@pytest.mark.parametrize("at", [
    (B0, None, B0, 1 << 24), (B0, None, B0 + 4092, 1 << 24), (B0, None, B0 - 252, 1 << 24),
    (B0, None, 1 << 24, B0 + 64), (B0, 1 << 24, (1 << 24) + 252, 1 << 25),
    (B0, 1 << 24, 1 << 25, (1 << 24) - 252), (B0, None, 1 << 24, (1 << 24) + 252),
    (B0, None, 1 << 24, 1 << 24),
])
def test_route_refuses_overlaps(at):
    assert _route(*at) == BAD


@pytest.mark.parametrize("act", [mb.ACT_NONE, mb.ACT_SWIGLU])
@pytest.mark.parametrize("q,qs,src", [
    (B0, 1 << 24, None), (1 << 24, B0, None), (B0 - 496, 1 << 24, None), (1 << 24, B0 + 1023, None),
    (1 << 24, (1 << 24) + 511, None), (1 << 24, 1 << 25, (1 << 24) + 508),
    (1 << 24, 1 << 25, (1 << 25) - 12),
])
def test_quantize_refuses_overlaps(q, qs, src, act):
    # x 2048 bytes (bf16; twice that in front of the activation), q 512, scales 32
    assert mb.raw_call("mb_quantize_mx4", 4, 256, mb.BF16, act, P(B0), P(src), P(q), P(qs),
                       None) == BAD


@pytest.mark.parametrize("x", [B0, B0 + 496, B0 - 2032, (1 << 24) + 16, (1 << 24) - 2032])
def test_dequantize_refuses_overlaps(x):
    assert mb.raw_call("mb_dequantize_mx4", 4, 256, mb.BF16, P(B0), P(1 << 24), P(x), None) == BAD


@pytest.mark.parametrize("kw", [
    dict(y=B0), dict(res=B0 + 16), dict(res=1 << 24, out=B0 + 16), dict(q=B0 + 2032),
    dict(y=1 << 24, q=(1 << 24) + 16), dict(qs=B0 + 4), dict(w=1 << 24, y=(1 << 24) + 496),
    dict(res=1 << 24, out=B0, y=B0), dict(res=1 << 24, out=1 << 24, q=1 << 24),
    dict(res=B0, out=B0, y=B0 + 16),
])
def test_norm_refuses_overlaps(kw):
    # rows of 2048 bytes (bf16), q 1024, scales 32, weight 512
    at = {**dict(res=None, w=1 << 27, out=None, y=None, q=1 << 28, qs=1 << 29), **kw}
    if kw == dict(res=B0 + 16):  # two inputs may overlap; the sum over one of them not
        at["out"] = B0
    assert mb.raw_call("mb_rmsnorm_fp8", 4, 256, mb.BF16, 1e-6, P(B0), P(at["res"]), P(at["w"]),
                       P(at["out"]), P(at["y"]), P(at["q"]), P(at["qs"]), None) == BAD


@pytest.mark.parametrize("name", ["a", "a_scale", "w", "w_scale", "cu_seqlens", "rep_expert",
                                  "status"])
@pytest.mark.parametrize("end", [False, True])
def test_expert_refuses_overlaps(name, end):
    d = _dims()
    names = ("a", "a_scale", "w", "w_scale", "cu_seqlens", "rep_expert", "status")
    at = {n: (i + 1) << 24 for i, n in enumerate(names)}
    rows, n, k = d.rows, 64, 128
    size = dict(a=rows * k // 2, a_scale=rows * k // 32, w=16 * n * k // 2, w_scale=16 * n * k // 32,
                cu_seqlens=4 * 6 * 4, rep_expert=4 * 4, status=16)[name]
    y = at[name] - rows * n * 2 + 16 if end else at[name] + (size - 1) // 16 * 16
    b = _bufs(**{f: at[f] for f in names[4:]})
    assert mb.raw_call("mb_expert_mx4", ctypes.byref(d), ctypes.byref(b), n, k,
                       *(P(at[f]) for f in names[:4]), P(y), None) == BAD
