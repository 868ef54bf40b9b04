"""Corners of the router, the norm, the 4-bit rows and their dispatch on the
GPU, each against its plain definition."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import token_dispatch_mb_amd as mb

from . import gpu_harness as G
from . import plain_ops as R
from .test_gpu_ops import check_route, dev, f64, rng

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
