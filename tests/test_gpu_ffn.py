"""The experts' products from bf16 rows, their gradients, the combine's
gradients and the projection with adapters on the GPU, against their plain
64-bit definitions and the error bounds derived there (``plain_ffn``)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import token_dispatch_mb_amd as mb
import workload as W

from . import gpu_harness as G
from . import plain_ffn as F
from . import plain_ops as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
MARK = -12345.0  # outputs hold it before the call


@pytest.fixture(autouse=True)
def _gpu_required():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def rng(*seed):
    return np.random.default_rng(seed)


def bf(r, *shape, std=1.0):
    """Normal bfloat16 values, as float64."""
    return R.bf16_round(np.float32(std * r.standard_normal(shape))).astype(np.float64)


def dev(a, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(G.dev())


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def out(*shape, dtype="bf16"):
    return torch.full(shape, MARK, dtype=DT[dtype], device=G.dev())


def marked(t):
    """Values that the call left as they were."""
    return f64(t) == float(torch.tensor(MARK, dtype=t.dtype))


def near(got, want, bound):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                           bound[bad][:4])


class Layer:
    """A plan with `rows` of every slot given, replicas of other ranks' experts
    in the replica slots, and `pad` rows behind a rank's last."""

    def __init__(self, counts, home, rep=None, pad=0, expected=None, dtype_out="bf16"):
        counts = np.asarray(counts)
        self.P, NS = counts.shape
        self.Eh, self.R = home, NS - home
        self.E, self.cap = self.P * home, int(counts.sum(axis=1).max()) + pad
        cu = np.zeros((self.P, NS + 1), np.int32)
        cu[:, 1:] = np.cumsum(counts, axis=1)
        if rep is None:  # replicas of the next rank's experts
            rep = [[((p + 1) % self.P) * home + i % home for i in range(self.R)] for p in range(self.P)]
        self.cu, self.rep = cu, np.array(rep, np.int32).reshape(self.P, self.R)
        n = int(counts.sum()) if expected is None else expected
        n = max(n // self.P, 1) * self.P
        self.dims = mb.Dims.make(n, 1, self.E, self.P, self.R, 128, cap=self.cap, dtype_out=dtype_out)
        self.bufs = mb.PlanBuffers.allocate(self.dims, G.dev())
        self.bufs.status.zero_()
        self.bufs.cu_seqlens = torch.from_numpy(cu).to(G.dev())
        self.bufs.rep_expert = torch.from_numpy(
            self.rep if self.R else np.full((self.P, 1), -1, np.int32)).to(G.dev())
        self.groups = R.slots(cu, self.rep, self.P, self.Eh, self.R, self.cap)
        self.used = np.zeros(self.P * self.cap, bool)
        for _, lo, hi in self.groups:
            self.used[lo:hi] = True

    @property
    def rows(self):
        return self.P * self.cap

    def tensor(self, a):
        """Rows on the GPU, with NaN where no slot's are."""
        t = dev(a)
        t[torch.from_numpy(~self.used).to(G.dev())] = float("nan")
        return t


SKEWED = [[37, 0, 5, 1], [0, 0, 130, 2], [3, 64, 0, 65]]  # three ranks, three experts and a replica
LAYERS = {
    "one_row": lambda **k: Layer([[1]], 1, **k),
    "sparse": lambda **k: Layer([[0, 1, 0], [2, 0, 0], [0, 0, 1], [0, 0, 0]], 2, pad=2, **k),
    "skewed": lambda **k: Layer(SKEWED, 3, pad=7, **k),
    "few": lambda **k: Layer(SKEWED, 3, pad=7, expected=12, **k),  # the kernel for few rows
    # a rank without replicas, an empty replica slot, an expert three times over
    "shared": lambda **k: Layer([[100, 40, 30], [0, 200, 0], [17, 70, 90]], 1, [[1, 1], [2, -1], [1, 0]],
                                pad=1, **k),
    "dense": lambda **k: Layer([[257, 700], [1024, 64]], 2, **k),
}
SIZES = [(8, 8), (16, 72), (72, 264), (264, 520), (520, 1032)]


def run_product(L, n, k, act, dtype, keep=True, seed=0):
    r = rng(n, k, seed)
    gated = act == "swiglu"
    a, w = bf(r, L.rows, k), bf(r, L.E, n * (2 if gated else 1), k, std=k**-0.5)
    y = out(L.rows, n, dtype=dtype)
    pre = out(L.rows, 2 * n) if gated and keep else None
    mb.expert_bf16(L.dims, L.bufs, n, k, L.tensor(a), dev(w), y, act=act, pre=pre)
    assert marked(y)[~L.used].all()
    got = f64(y)
    gp = None if pre is None else f64(pre)
    for e, lo, hi in L.groups:
        if gated:
            g, eg, u, eu, h, eh = F.gated(a[lo:hi], w[e])
            near(got[lo:hi], h, F.rounded(h, eh, dtype))
            if keep:
                near(gp[lo:hi, :n], g, F.rounded(g, eg, "bf16"))
                near(gp[lo:hi, n:], u, F.rounded(u, eu, "bf16"))
        else:
            v, e = F.product(a[lo:hi], w[e])
            near(got[lo:hi], v, F.rounded(v, e, dtype))
    if keep and gated:
        assert marked(pre)[~L.used].all()


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("layer", LAYERS)
def test_product(layer, n, k):
    run_product(LAYERS[layer](), n, k, "none", "bf16")
    run_product(LAYERS[layer](dtype_out="f32"), n, k, "none", "f32")


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("layer", LAYERS)
def test_gated_product(layer, n, k):
    run_product(LAYERS[layer](), n, k, "swiglu", "bf16")
    run_product(LAYERS[layer](dtype_out="f32"), n, k, "swiglu", "bf16", keep=False)


def run_dgrad(L, n, k, act, dtype):
    r = rng(n, k, 1)
    gated = act == "swiglu"
    dy, w = bf(r, L.rows, n), bf(r, L.E, n, k, std=n**-0.5)
    pre = 3 * bf(r, L.rows, 2 * k) if gated else None
    pre = None if pre is None else R.bf16_round(np.float32(pre)).astype(np.float64)
    da = out(L.rows, k * (2 if gated else 1), dtype=dtype)
    mb.expert_bf16_dgrad(L.dims, L.bufs, n, k, L.tensor(dy), dev(w), da, act=act,
                         pre=None if pre is None else L.tensor(pre))
    assert marked(da)[~L.used].all()
    got = f64(da)
    for e, lo, hi in L.groups:
        if gated:
            dg, eg, du, eu = F.gate_grad(dy[lo:hi], w[e], pre[lo:hi, :k], pre[lo:hi, k:])
            near(got[lo:hi, :k], dg, F.rounded(dg, eg, "bf16"))
            near(got[lo:hi, k:], du, F.rounded(du, eu, "bf16"))
        else:
            v, e = F.row_grad(dy[lo:hi], w[e])
            near(got[lo:hi], v, F.rounded(v, e, dtype))


@pytest.mark.parametrize("n,k", [(k, n) for n, k in SIZES] + [(264, 72)])
@pytest.mark.parametrize("layer", LAYERS)
def test_row_gradients(layer, n, k):
    run_dgrad(LAYERS[layer](), n, k, "none", "bf16")
    run_dgrad(LAYERS[layer](dtype_out="f32"), n, k, "none", "f32")
    run_dgrad(LAYERS[layer](), n, k, "swiglu", "bf16")


def run_wgrad(L, n, k, dtype, add):
    r = rng(n, k, 2)
    dy, a = bf(r, L.rows, n), bf(r, L.rows, k)
    dw = out(L.E, n, k, dtype=dtype)
    old = np.zeros((L.E, n, k))
    if add:
        old = bf(r, L.E, n, k)
        dw.copy_(dev(old, DT[dtype]))
    mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, L.tensor(dy), L.tensor(a), dw, accumulate=add)
    got = f64(dw)
    for e in range(L.E):
        rows = np.concatenate([np.arange(lo, hi) for x, lo, hi in L.groups if x == e] +
                              [np.zeros(0, int)]).astype(int)
        v, err = F.weight_grad(dy[rows], a[rows])
        v, err = v + old[e], err + 2.0**-23 * (np.abs(old[e]) + np.abs(v))
        near(got[e], v, F.rounded(v, err, dtype))


@pytest.mark.parametrize("n,k", SIZES + [(1032, 264)])
@pytest.mark.parametrize("layer", LAYERS)
def test_weight_gradients(layer, n, k):
    L = LAYERS[layer]()
    for dtype in ("f32", "bf16"):
        run_wgrad(L, n, k, dtype, add=False)
        run_wgrad(L, n, k, dtype, add=True)


@pytest.mark.parametrize("counts", [[[4000]], [[1500, 250, 1300, 1000]], [[700, 385, 513, 64] * 2]])
def test_whole_tiles(counts):
    """Sizes that take tiles of 256 rows, in a product, its gradients, and both
    reductions; every number of rows left over in a tile."""
    home = len(counts[0])
    L = Layer(counts, home, pad=1, dtype_out="f32")
    n, k = 4104, 72
    run_product(L, n, k, "none", "f32")
    run_product(L, n, k, "swiglu", "bf16")
    run_dgrad(L, k, n, "none", "f32")
    run_dgrad(L, k, n, "swiglu", "bf16")
    L = Layer(counts, home, pad=1)
    run_product(L, n, k, "none", "bf16")
    run_dgrad(L, k, n, "none", "bf16")
    n, k = 1288, 1544
    for dtype in ("f32", "bf16"):
        run_wgrad(Layer(np.asarray(counts) // 4, home), 2 * n, 2 * k, dtype, add=dtype == "f32")


def test_many_slots():
    """1024 experts and 1024 replica slots, most of them empty."""
    r = rng(9)
    counts = np.where(r.random((64, 32)) < 0.1, r.integers(1, 4, (64, 32)), 0)
    rep = r.integers(-1, 1024, (64, 16))
    L = Layer(counts, 16, rep, pad=1)
    run_product(L, 72, 40, "none", "bf16")
    run_product(L, 72, 40, "swiglu", "bf16")
    run_dgrad(L, 40, 72, "none", "bf16")
    run_wgrad(L, 24, 40, "f32", add=False)


def test_far_gates_keep_their_value():
    """silu(g) of gates where exp(-g) passes binary32, and its gradients; an
    infinite gate gives what the formula gives, and only in its own output."""
    L = Layer([[64]], 1)
    k = n = 64
    gates = np.float64([-200, -120, -104, -100, -90, -88.5, -87, -80.5, -60, -20, 0, 20, 88, 90, 120, 2000])
    a = np.zeros((64, k))
    a[np.arange(64), np.arange(64)] = 1
    w = np.zeros((1, 2 * n, k))
    w[0, :n] = gates[np.arange(n) % 16][:, None]
    w[0, n:] = 2.0
    y, pre = out(64, n), out(64, 2 * n)
    for few in (False, True):
        d = L.dims if not few else mb.Dims.make(1, 1, 1, 1, 0, 128, cap=64)
        mb.expert_bf16(d, L.bufs, n, k, dev(a), dev(w), y, act="swiglu", pre=pre)
        g = R.bf16_round(np.float32(w[0, :n, 0])).astype(np.float64)
        h = g * F.sigmoid(g) * 2
        near(f64(y), np.broadcast_to(h, (64, n)), np.broadcast_to(
            F.rounded(h, np.abs(h) * (F.sigmoid_error(g) + 2.0**-21), "bf16"), (64, n)))
    dy = np.zeros((64, k))
    dy[np.arange(64), np.arange(64)] = 1
    eye = np.eye(64)[None] * 4.0
    da = out(64, 2 * n)
    p = np.concatenate((np.broadcast_to(g, (64, n)), np.full((64, n), 0.5)), axis=1)
    mb.expert_bf16_dgrad(L.dims, L.bufs, k, n, dev(dy), dev(eye), da, act="swiglu", pre=dev(p))
    dg, eg, du, eu = F.gate_grad(dy, eye[0], p[:, :n], p[:, n:])
    near(f64(da)[:, :n], dg, F.rounded(dg, eg, "bf16"))
    near(f64(da)[:, n:], du, F.rounded(du, eu, "bf16"))


def test_infinities_and_nan_stay_in_their_rows_and_columns():
    L = Layer([[40, 3]], 2)
    n, k = 24, 88
    r = rng(5)
    a, w = bf(r, L.rows, k), bf(r, 2, n, k)
    a[7, 80], w[0, 5, 3], a[41, 0] = np.nan, np.inf, -np.inf
    for exp in (43, 2):
        d = mb.Dims.make(exp, 1, 2, 1, 0, 128, cap=L.cap, dtype_out="f32")
        y = out(L.rows, n, dtype="f32")
        mb.expert_bf16(d, L.bufs, n, k, dev(a), dev(w), y)
        got = f64(y)
        want = np.ones(got.shape, bool)
        want[7], want[:40, 5], want[41] = False, False, False
        assert np.array_equal(np.isfinite(got), want)
    dw = out(2, n, k, dtype="f32")
    dy = bf(r, L.rows, n)
    dy[12, 4] = np.nan
    mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, dev(dy), dev(bf(r, L.rows, k)), dw)
    want = np.ones((2, n, k), bool)
    want[0, 4] = False
    assert np.array_equal(np.isfinite(f64(dw)), want)


def test_a_fatal_status_leaves_everything():
    L = LAYERS["skewed"]()
    L.bufs.status[0] = mb.ST_CAPACITY
    n, k = 64, 72
    r = rng(1)
    y, da, dw = out(L.rows, n), out(L.rows, k), out(L.E, n, k)
    a, w, dy = dev(bf(r, L.rows, k)), dev(bf(r, L.E, n, k)), dev(bf(r, L.rows, n))
    mb.expert_bf16(L.dims, L.bufs, n, k, a, w, y)
    few = mb.Dims.make(3, 1, L.E, L.P, L.R, 128, cap=L.cap)
    mb.expert_bf16(few, L.bufs, n, k, a, w, y)
    mb.expert_bf16_dgrad(L.dims, L.bufs, n, k, dy, w, da)
    mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, dy, a, dw)
    for t in (y, da, dw):
        assert marked(t).all()


def test_wgrad_without_tokens_gives_zeros():
    d = mb.Dims.make(0, 2, 6, 3, 1, 128, cap=4)
    bufs = mb.PlanBuffers.allocate(d, G.dev())
    mb.plan(d, torch.zeros(0, dtype=torch.int32, device=G.dev()), mb.alloc_workspace(d, G.dev()), bufs)
    a = torch.full((12, 40), float("nan"), dtype=torch.bfloat16, device=G.dev())
    dw = out(6, 40, 40)
    mb.expert_bf16_wgrad(d, bufs, 40, 40, a, a, dw)
    assert not f64(dw).any()
    dw = out(6, 40, 40)
    mb.expert_bf16_wgrad(d, bufs, 40, 40, a, a, dw, accumulate=True)
    assert marked(dw).all()


# ------------------------------------------------------------ combine's gradients

@pytest.mark.parametrize("n,k,h,dtype", [
    (1, 1, 4, "f32"), (1, 1, 8, "bf16"), (3, 2, 128, "bf16"), (77, 6, 1032, "bf16"), (33, 32, 264, "f32"),
    (130, 8, 7168, "bf16"), (65, 4, 516, "f32"), (9, 3, 4104, "bf16"), (200, 2, 4096, "f32"),
    (500, 8, 512, "bf16"),
])
def test_combine_gradients(n, k, h, dtype):
    r = rng(n, k, h)
    d = mb.Dims.make(n, k, max(k, 2), 1, 0, h, cap=n * k + 3, dtype_in=dtype, dtype_out=dtype)
    bufs = mb.PlanBuffers.allocate(d, G.dev())
    pos = r.permutation(n * k + 3)[: n * k].reshape(n, k)
    bufs.pos = torch.from_numpy(pos.astype(np.int32)).to(G.dev())
    bufs.status.zero_()
    dy, ye = bf(r, n, h), bf(r, d.rows, h)
    w = np.float32(r.standard_normal((n, k))).astype(np.float64)
    rows, dw, err = F.combine_grad(pos, w, dy, ye)
    D, Y, Wt = dev(dy, DT[dtype]), dev(ye, DT[dtype]), dev(w, torch.float32)
    for which in ("both", "rows", "weights"):
        go, gw = out(d.rows, h, dtype=dtype), out(n, k, dtype="f32")
        mb.combine_grad(d, bufs, D, Y if which != "rows" else None, Wt if which != "weights" else None,
                        go if which != "weights" else None, gw if which != "rows" else None)
        if which != "weights":
            near(f64(go)[pos], rows, F.rounded(rows, np.abs(rows) * 2.0**-24, dtype))
            rest = np.ones(d.rows, bool)
            rest[pos.ravel()] = False
            assert marked(go)[rest].all()
        else:
            assert marked(go).all()
        if which != "rows":
            near(f64(gw), dw, F.rounded(dw, err, "f32"))
        else:
            assert marked(gw).all()


def test_combine_gradients_of_a_broken_or_fatal_plan():
    d = mb.Dims.make(4, 2, 2, 1, 0, 64, cap=8)
    bufs = mb.PlanBuffers.allocate(d, G.dev())
    bufs.status.zero_()
    bufs.pos = torch.tensor([[0, 1], [-1, 8], [2**31 - 1, 3], [4, -2**31]], dtype=torch.int32,
                            device=G.dev())
    r = rng(2)
    dy, ye, w = bf(r, 4, 64), bf(r, 8, 64), bf(r, 4, 2)
    go, gw = out(8, 64), out(4, 2, dtype="f32")
    mb.combine_grad(d, bufs, dev(dy), dev(ye), dev(w, torch.float32), go, gw)
    assert marked(go)[[2, 5, 6, 7]].all() and not marked(go)[[0, 1, 3, 4]].any()
    g = f64(gw)
    assert (g[[1, 1, 2, 3], [0, 1, 0, 1]] == 0).all()  # pairs without a row
    near(g[0], ye[[0, 1]] @ dy[0], np.full(2, 1e-3))
    bufs.status[0] = mb.ST_DUP_ID
    go, gw = out(8, 64), out(4, 2, dtype="f32")
    mb.combine_grad(d, bufs, dev(dy), dev(ye), dev(w, torch.float32), go, gw)
    assert marked(go).all() and marked(gw).all()


# ------------------------------------------------------------ adapters

def run_lora(t, n, k, rank, L, adapter, dtype, seed=0, stream=None):
    r = rng(t, n, k, rank, seed)
    x, w = bf(r, t, k), bf(r, n, k, std=k**-0.5)
    a, b = bf(r, L, rank, k, std=k**-0.5), bf(r, L, n, rank, std=rank**-0.5)
    scale = np.float32(0.5 + r.random(L)).astype(np.float64)
    prm = mb.LoraParams.make(t, n, k, rank, L, dtype_out=dtype)
    ws = mb.alloc_lora_workspace(prm, G.dev())
    ws.fill_(0xFF)  # NaN: nothing may be read before it is written
    y = out(t, n, dtype=dtype)
    ad = torch.from_numpy(np.asarray(adapter, np.int32)).to(G.dev())
    mb.project_lora(prm, dev(x), dev(w), dev(a), dev(b), dev(scale, torch.float32), ad, ws, y)
    want, err = F.lora(x, w, a, b, scale, adapter)
    near(f64(y), want, F.rounded(want, err, dtype))


LORA = [  # rows, outputs, terms, rank, adapters
    (1, 8, 8, 8, 1), (1, 264, 1032, 16, 3), (5, 72, 136, 24, 7), (16, 520, 2056, 16, 40),
    (17, 520, 2056, 16, 40), (33, 8, 264, 8, 2), (64, 1032, 520, 32, 9), (100, 264, 4104, 40, 30),
    (129, 776, 776, 16, 5), (257, 520, 264, 256, 3), (300, 2056, 72, 8, 11), (700, 264, 1032, 48, 6),
    (4400, 4360, 72, 16, 9), (4400, 4360, 136, 40, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,n,k,rank,L", LORA)
def test_lora(t, n, k, rank, L, dtype):
    r = rng(t, n)
    mixed = r.integers(-1, L, t)
    runs = np.sort(mixed)[r.permutation(t) if t < 8 else np.arange(t)]
    run_lora(t, n, k, rank, L, mixed, dtype)
    if t > 1:
        run_lora(t, n, k, rank, L, runs, dtype, seed=1)


@pytest.mark.parametrize("t", [1, 16, 50, 300, 4400])
def test_lora_numbers_that_are_no_adapter(t):
    r = rng(t)
    odd = np.array([-1, 3, 2**31 - 1, -2**31, 0, 2])
    run_lora(t, 4360 if t > 1000 else 72, 72, 16, 3, odd[r.integers(0, 6, t)], "f32")
    run_lora(t, 4360 if t > 1000 else 72, 72, 16, 3, np.full(t, -1), "bf16")


@pytest.mark.parametrize("t", [4, 40, 4400])
def test_lora_infinities_and_nan_stay_in_their_rows(t):
    n, k = (4360 if t > 1000 else 72), 72
    r = rng(t)
    x, w, a, b = bf(r, t, k), bf(r, n, k), bf(r, 2, 8, k), bf(r, 2, n, 8)
    a[1, 3, 5], b[1, 3, 2] = np.inf, -np.inf
    x[2, 7] = np.nan
    ad = np.arange(t, dtype=np.int32) % 3 - 1  # none, 0, 1 by turns
    prm = mb.LoraParams.make(t, n, k, 8, 2, dtype_out="f32")
    y = out(t, n, dtype="f32")
    mb.project_lora(prm, dev(x), dev(w), dev(a), dev(b), dev(np.ones(2), torch.float32),
                    torch.from_numpy(ad).to(G.dev()), mb.alloc_lora_workspace(prm, G.dev()), y)
    bad = (ad == 1) | (np.arange(t) == 2)
    assert np.array_equal(np.isfinite(f64(y)).all(axis=1), ~bad)


def test_lora_calls_on_two_streams_at_once():
    r = rng(8)
    sizes = [(40, 264, 1032), (300, 520, 776)]
    args, want = [], []
    for t, n, k in sizes:
        prm = mb.LoraParams.make(t, n, k, 16, 4, dtype_out="f32")
        v = [dev(bf(r, t, k)), dev(bf(r, n, k)), dev(bf(r, 4, 16, k)), dev(bf(r, 4, n, 16)),
             dev(np.ones(4), torch.float32),
             torch.from_numpy(r.integers(-1, 4, t).astype(np.int32)).to(G.dev())]
        y = out(t, n, dtype="f32")
        mb.project_lora(prm, *v, mb.alloc_lora_workspace(prm, G.dev()), y)
        args.append((prm, v, mb.alloc_lora_workspace(prm, G.dev())))
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [torch.full_like(y, MARK) for y in want]
        torch.cuda.synchronize()
        for (prm, v, ws), y, st in zip(args, got, streams):
            mb.project_lora(prm, *v, ws, y, stream=st)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------ a layer's training step

class Step:
    """A layer's forward and backward pass: plan, dispatch, both products,
    combine, and the gradients of its input, weights and gate weights."""

    def __init__(self, P=4, E=8, N=96, K=2, H=264, I=136, seed=0):
        r = rng(seed, N, H)
        self.N, self.K, self.H, self.I, self.E = N, K, H, I, E
        self.d = mb.Dims.make(N, K, E, P, 1, H, cap=3 * N * K // P)
        pick = np.argsort(r.random((N, E)) - 0.7 * (np.arange(E) < 2), axis=1)[:, :K]
        self.ids, self.x = pick.astype(np.int32), bf(r, N, H)
        self.gate = np.float32(r.random((N, K)) + 0.1).astype(np.float64)
        self.w1, self.w2 = bf(r, E, 2 * I, H, std=H**-0.5), bf(r, E, H, I, std=I**-0.5)
        self.dy = bf(r, N, H)
        g = G.dev()
        self.t = {n: dev(getattr(self, n)) for n in ("x", "w1", "w2", "dy")}
        self.t["ids"] = torch.from_numpy(self.ids).to(g)
        self.t["gate"] = dev(self.gate, torch.float32)
        self.t["one"] = torch.ones(N, K, device=g)
        self.bufs, self.ws = mb.PlanBuffers.allocate(self.d, g), mb.alloc_workspace(self.d, g)
        M = self.d.rows
        e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=g)  # noqa: E731
        self.o = {"buf": e(M, H), "mid": e(M, I), "pre": e(M, 2 * I), "ye": e(M, H), "y": e(N, H),
                  "dye": e(M, H), "dgate": e(N, K, dt=torch.float32), "dpre": e(M, 2 * I),
                  "dbuf": e(M, H), "dx": e(N, H), "dw1": e(E, 2 * I, H, dt=torch.float32),
                  "dw2": e(E, H, I, dt=torch.float32)}

    def run(self, stream=None):
        d, b, t, o, H, I = self.d, self.bufs, self.t, self.o, self.H, self.I
        mb.plan(d, t["ids"], self.ws, b, stream)
        mb.dispatch(d, b, t["x"], o["buf"], stream=stream)
        mb.expert_bf16(d, b, I, H, o["buf"], t["w1"], o["mid"], act="swiglu", pre=o["pre"], stream=stream)
        mb.expert_bf16(d, b, H, I, o["mid"], t["w2"], o["ye"], stream=stream)
        mb.combine(d, b, o["ye"], t["gate"], o["y"], stream=stream)
        mb.combine_grad(d, b, t["dy"], o["ye"], t["gate"], o["dye"], o["dgate"], stream=stream)
        mb.expert_bf16_dgrad(d, b, H, I, o["dye"], t["w2"], o["dpre"], act="swiglu", pre=o["pre"],
                             stream=stream)
        mb.expert_bf16_wgrad(d, b, H, I, o["dye"], o["mid"], o["dw2"], stream=stream)
        mb.expert_bf16_dgrad(d, b, 2 * I, H, o["dpre"], t["w1"], o["dbuf"], stream=stream)
        mb.expert_bf16_wgrad(d, b, 2 * I, H, o["dpre"], o["buf"], o["dw1"], stream=stream)
        mb.combine(d, b, o["dbuf"], t["one"], o["dx"], stream=stream)  # the dispatch's gradient

    def exact(self):
        """The layer and its gradients by automatic differentiation in 64 bits."""
        T = lambda a: torch.tensor(a, dtype=torch.float64, requires_grad=True)  # noqa: E731
        x, gate, w1, w2 = T(self.x), T(self.gate), T(self.w1), T(self.w2)
        y = torch.zeros(self.N, self.H, dtype=torch.float64)
        for k in range(self.K):
            i = torch.from_numpy(self.ids[:, k]).long()
            pre = torch.matmul(w1[i], x[:, :, None])[:, :, 0]
            mid = torch.nn.functional.silu(pre[:, : self.I]) * pre[:, self.I:]
            y = y + gate[:, k:k + 1] * torch.matmul(w2[i], mid[:, :, None])[:, :, 0]
        (y * torch.tensor(self.dy)).sum().backward()
        return {"y": y, "dx": x.grad, "dgate": gate.grad, "dw1": w1.grad, "dw2": w2.grad}


def test_a_training_step():
    """Every output within the roundings that lie between: rows are rounded to
    bfloat16 (2^-8 each, independent, so a sum of many is off by about 2^-8 of
    its root of squares) three times on the way to y, at most five to dx and
    dw1. 12 of them for the largest of 25000 values: 12 * 2^-8 of the root mean
    square and of the value."""
    s = Step()
    s.run()
    assert mb.plan_status(s.bufs)[0] & mb.ST_FATAL == 0
    for name, want in s.exact().items():
        want, got = want.detach().numpy(), f64(s.o[name])
        rms = np.sqrt((want**2).mean())
        near(got, want, 12 * 2.0**-8 * (rms + np.abs(want)))


def test_a_training_step_captured_and_replayed():
    s = Step(N=200, H=520, I=264, seed=3)
    s.run()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in s.o.items()}
    used = (s.bufs.row_src >= 0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        s.run(st)
    for _ in range(4):
        for v in s.o.values():
            v.fill_(MARK)
        (want["y"].float() @ want["y"].float().t()).sum().item()  # other work between replays
        g.replay()
        torch.cuda.synchronize()
        for k, v in s.o.items():
            rows = v.shape[0] == s.d.rows  # rows of no slot are left as they were
            assert torch.equal(v[used] if rows else v, want[k][used] if rows else want[k]), k


def test_a_step_on_another_stream():
    s = Step(seed=5)
    s.run()
    torch.cuda.synchronize()
    want = {k: s.o[k].clone() for k in ("y", "dx", "dgate", "dw1", "dw2")}
    for k in want:
        s.o[k].fill_(MARK)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    s.run(st)
    st.synchronize()
    for k, v in want.items():
        assert torch.equal(s.o[k], v), k


# ------------------------------------------------------------ what the binding refuses

def test_binding_checks():
    L = LAYERS["skewed"]()
    n, k = 64, 72
    a, w = out(L.rows, k), out(L.E, n, k)
    y = out(L.rows, n)
    with pytest.raises(TypeError):
        mb.expert_bf16(L.dims, L.bufs, n, k, a.float(), w, y)
    with pytest.raises(TypeError):
        mb.expert_bf16(L.dims, L.bufs, n, k, a, w, y.float())
    with pytest.raises(ValueError, match="elements"):
        mb.expert_bf16(L.dims, L.bufs, n, k, a, w[:-1], y)
    with pytest.raises(ValueError, match="elements"):
        mb.expert_bf16(L.dims, L.bufs, n, k, a, w, y, act="swiglu")
    with pytest.raises(ValueError, match="contiguous"):
        mb.expert_bf16(L.dims, L.bufs, n, k, a, w.transpose(1, 2), y)
    with pytest.raises(ValueError, match="overlap"):
        mb.expert_bf16(L.dims, L.bufs, k, k, a, out(L.E, k, k), a)
    with pytest.raises(mb.MoebalError):
        mb.expert_bf16(L.dims, L.bufs, n, k, a, w, y, pre=out(L.rows, 2 * n))
    with pytest.raises(mb.MoebalError):
        mb.expert_bf16_dgrad(L.dims, L.bufs, n, k, y, w, out(L.rows, 2 * k), act="swiglu")
    with pytest.raises(TypeError):
        mb.expert_bf16_wgrad(L.dims, L.bufs, n, k, y, a, out(L.E, n, k).half())
    # dw begins where dy does
    big = out(max(L.rows * n, L.E * n * n))
    with pytest.raises(ValueError, match="overlap"):
        mb.expert_bf16_wgrad(L.dims, L.bufs, n, n, big[: L.rows * n], y, big)


# ------------------------------------------------------------ both sides of what picks a kernel

@pytest.mark.parametrize("counts", [[[3830]], [[1400, 250, 1200, 700]], [[600, 385, 513, 64] * 2]])
def test_one_round_of_tall_tiles(counts):
    """Tiles of 256 rows that fill the CUs once, of 128 rows twice."""
    home = len(counts[0])
    n, k = 4104, 72
    for dtype in ("f32", "bf16"):
        L = Layer(counts, home, pad=1, dtype_out=dtype)
        run_product(L, n, k, "none", dtype)
        run_dgrad(L, k, n, "none", dtype)
    run_dgrad(L, k, n, "swiglu", "bf16")
    run_product(L, 2056, k, "swiglu", "bf16")


@pytest.mark.parametrize("rows", [7, 8, 9, 40])
def test_rows_in_a_slot_around_the_kernel_for_few(rows):
    """The same slots, some with far more rows than expected."""
    for counts in ([[rows] * 3, [rows, 0, 2 * rows]], [[6 * rows, 0, 0], [0, 0, 0]]):
        L = Layer(counts, 3, pad=2)
        run_product(L, 264, 520, "swiglu", "bf16")
        run_product(L, 72, 1032, "none", "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,n,k,rank,L", [
    (3830, 4104, 72, 16, 9),  # tall tiles, the reduction in one
    (130, 16648, 2000, 16, 9),  # tall tiles, in three parts
    (100, 1032, 4104, 40, 30), (256, 520, 2056, 256, 4),  # low tiles in parts
    (300, 520, 136, 16, 5),  # low tiles, the reduction in one
    (48, 1032, 520, 24, 6), (48, 1352, 520, 24, 6),  # few rows, and past them
])
def test_lora_shapes(t, n, k, rank, L, dtype):
    r = rng(t, n)
    run_lora(t, n, k, rank, L, r.integers(-1, L, t), dtype)
    run_lora(t, n, k, rank, L, np.arange(t) // 60 % (L + 1) - 1, dtype, seed=1)


@pytest.mark.parametrize("t,n,k", [(64, 1032, 1032), (3830, 4104, 72)])
def test_lora_infinities_in_one_adapter(t, n, k):
    r = rng(t)
    x, w, a, b = bf(r, t, k), bf(r, n, k), bf(r, 2, 8, k), bf(r, 2, n, 8)
    a[1, 3, 5], b[1, 3, 2] = np.inf, np.nan
    ad = np.arange(t, dtype=np.int32) % 3 - 1  # none, 0, 1 by turns
    prm = mb.LoraParams.make(t, n, k, 8, 2, dtype_out="f32")
    y = out(t, n, dtype="f32")
    mb.project_lora(prm, dev(x), dev(w), dev(a), dev(b), dev(np.ones(2), torch.float32),
                    torch.from_numpy(ad).to(G.dev()), mb.alloc_lora_workspace(prm, G.dev()), y)
    good = np.isfinite(f64(y))
    assert good[ad != 1].all()
    assert not good[ad == 1].any()
