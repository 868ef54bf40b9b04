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
