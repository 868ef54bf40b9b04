"""Measured cases of the experts' feed-forward block, its gradients, the
combine's gradient and the projections with adapters.

Each operator in a plain form of elementary torch operations (``own`` false)
and through this library (``own`` true):

* ffn  — the experts' gated feed-forward block over the dispatch buffer, bf16
  rows and weights: both projections with silu(gate) * up, then the product
  back to the rows' width; in training the projections and the activation are
  kept;
* grad — the gradients of the whole block (of its rows and of both weights; an
  expert's replicas add up), or of one product in fp32;
* comb — the gradients of the combine: of the experts' outputs and of the gate
  weights;
* lora — a shared projection with the low-rank adapters of many requests.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one step of a small model's layer: nothing but latency
        _ffn("ffn_tiny", rows=16, ranks=8, home=1, slots=1, hidden=1024, inner=512),
        # a decode batch: two rows for each of 64 experts, the weights stream through once
        _ffn("ffn_decode", rows=128, ranks=16, home=4, slots=1, hidden=7168, inner=2048),
        # 4096 tokens of an 8-expert top-2 layer, kept for its gradients, regions with rows to spare
        _ffn("ffn_8experts", rows=8192, ranks=8, home=1, slots=1, hidden=4096, inner=14336,
             train=True, pad=128),
        # a prefill batch over 256 experts on 32 ranks
        _ffn("ffn_prefill", rows=131072, ranks=32, home=8, slots=1, hidden=7168, inner=2048),
        # odd sizes, few rows: some experts get none
        _grad("grad_odd", rows=60, ranks=4, home=6, slots=2, hidden=1048, inner=328, pad=3),
        # the 8-expert layer's backward pass
        _grad("grad_8experts", rows=8192, ranks=8, home=1, slots=1, hidden=4096, inner=14336),
        # one product's gradients over 64 experts, in fp32
        _grad("grad_product", rows=65536, ranks=16, home=4, slots=1, hidden=7168, inner=2048,
              block=False),
        # 4096 tokens, two experts each, fp32 rows
        _comb("comb_top2", tokens=4096, k=2, hidden=4096, dtype="f32"),
        # a training batch with eight experts to a token, bf16 rows
        _comb("comb_top8", tokens=32768, k=8, hidden=7168, dtype="bf16"),
        # one token of one request
        _lora("lora_token", tokens=1, n=4096, k=4096, rank=16, adapters=8, requests=1),
        # a decode batch, every request with an adapter of its own
        _lora("lora_decode", tokens=64, n=7168, k=7168, rank=16, adapters=64, requests=64),
        # a prefill batch of a dozen prompts
        _lora("lora_prefill", tokens=16384, n=7168, k=7168, rank=32, adapters=16, requests=12),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("ffn", "grad", "comb", "lora"))
    if op == "comb":
        k = rng.choice((1, 2, 2, 4, 6, 8, 8, 10))
        return _comb(None, tokens=log_int(1, 200000 // k), k=k, hidden=8 * log_int(16, 1000),
                     dtype=rng.choice(("bf16", "bf16", "f32")))
    if op == "lora":
        tokens = log_int(1, 16384)
        return _lora(None, tokens=tokens, n=8 * log_int(32, 896), k=8 * log_int(32, 896),
                     rank=rng.choice((8, 16, 16, 24, 32)), adapters=log_int(1, 64),
                     requests=min(tokens, log_int(1, 200)), out=rng.choice(("bf16", "bf16", "f32")))
    ranks, home = rng.choice(((1, 1), (1, 8), (8, 1), (3, 5), (8, 4), (16, 4)))
    sizes = dict(rows=ranks * log_int(1, 40000 // ranks), ranks=ranks, home=home,
                 slots=rng.choice((0, 1, 2)), pad=rng.choice((0, 0, 5, 64)),
                 hidden=8 * log_int(16, 896), inner=8 * log_int(8, 400))
    if op == "ffn":
        return _ffn(None, train=rng.random() < 0.5, **sizes)
    return _grad(None, block=rng.random() < 0.6, **sizes)


def _named(name, case):
    return case if name is None else dict(case, name=name)


def _ffn(name, rows, ranks, home, slots, hidden, inner, train=False, pad=0):
    return _named(name, dict(op="ffn", rows=rows, ranks=ranks, home=home, slots=slots,
                             hidden=hidden, inner=inner, train=train, pad=pad))


def _grad(name, rows, ranks, home, slots, hidden, inner, block=True, pad=0):
    return _named(name, dict(op="grad", rows=rows, ranks=ranks, home=home, slots=slots,
                             hidden=hidden, inner=inner, block=block, pad=pad))


def _comb(name, tokens, k, hidden, dtype):
    return _named(name, dict(op="comb", tokens=tokens, k=k, hidden=hidden, dtype=dtype))


def _lora(name, tokens, n, k, rank, adapters, requests, out="bf16"):
    return _named(name, dict(op="lora", tokens=tokens, n=n, k=k, rank=rank, adapters=adapters,
                             requests=requests, out=out))


def work(case):
    op = case["op"]
    if op == "comb":
        t, k, h = case["tokens"], case["k"], case["hidden"]
        b = 4 if case["dtype"] == "f32" else 2
        return {"bytes": t * h * b * (1 + 2 * k) + t * k * 12, "flops": 3 * t * k * h}
    if op == "lora":
        t, n, k, r = case["tokens"], case["n"], case["k"], case["rank"]
        # a request of six has no adapter
        used = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** (case["requests"] * 5 / 6))
        return {"bytes": 2 * n * k + 2 * t * k + t * n * (4 if case["out"] == "f32" else 2) +
                int(2 * used * r * (n + k)) + 4 * t,
                "flops": 2 * t * n * k + int(5 / 6 * 2 * t * r * (n + k))}
    rows, h, i = case["rows"], case["hidden"], case["inner"]
    slots = case["ranks"] * (case["home"] + case["slots"])
    experts = case["ranks"] * case["home"]
    used = min(experts, slots * (1 - math.exp(-rows / slots)))  # experts that get a row at all
    if op == "ffn":
        # rows in and out, both weights; in training the projections and the activation
        keep = rows * 3 * i * 2 if case["train"] else 0
        return {"bytes": int(rows * h * 4 + used * 3 * i * h * 2 + keep), "flops": 6 * rows * h * i}
    if case["block"]:
        # x, dy, the projections and the activation in, dx out; weights in, their gradients out
        return {"bytes": int(rows * (3 * h + 3 * i) * 2 + (used + experts) * 3 * i * h * 2),
                "flops": 12 * rows * h * i}
    # dy, a in, da out; weights in, their gradients out
    return {"bytes": int(rows * (h + i) * 2 + rows * i * 4 + (2 * used + 4 * experts) * i * h),
            "flops": 4 * rows * h * i}


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case, "kept": {}}
    {"ffn": _prepare_ffn, "grad": _prepare_grad, "comb": _prepare_comb,
     "lora": _prepare_lora}[case["op"]](case, g, s)
    return s


def _randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    """Normal values, made a piece at a time (the weights are large)."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.normal_(0.0, std, generator=g)
    return out


def _prepare_plan(case, g, s):
    """The plan of the layer: replicas of experts homed elsewhere, some slots
    empty, rows skewed over the slots of a rank, `pad` rows behind the last."""
    P, Eh, R = case["ranks"], case["home"], case["slots"]
    E, NS, used = P * Eh, Eh + R, case["rows"] // P
    cap = used + case["pad"]
    rep = torch.randint(0, E, (P, max(R, 1)), generator=g, device="cuda", dtype=torch.int32)
    at = torch.arange(P, device="cuda", dtype=torch.int32)[:, None]
    drop = (rep // Eh == at) | (torch.rand(rep.shape, generator=g, device="cuda") < 0.2)
    rep = torch.where(drop, torch.full_like(rep, -1), rep)
    share = torch.rand((P, NS), generator=g, device="cuda") ** 2 + 0.05
    if R:
        share[:, Eh:] = torch.where(rep < 0, torch.zeros_like(share[:, Eh:]), share[:, Eh:])
    cdf = torch.cumsum(share, 1)
    cdf = cdf / cdf[:, -1:]
    u = torch.rand((P, used), generator=g, device="cuda")
    below = (u[:, :, None] >= cdf[:, None, :-1]).sum(2, dtype=torch.int64)
    count = torch.zeros((P, NS), dtype=torch.int64, device="cuda").scatter_add_(
        1, below, torch.ones_like(below))
    cu = torch.zeros((P, NS + 1), dtype=torch.int32, device="cuda")
    cu[:, 1:] = torch.cumsum(count, 1).int()
    s["cap"], s["cu"], s["rep"] = cap, cu, rep
    # the same plan as a host program that walks the groups keeps it
    cu_h, rep_h = cu.tolist(), rep.tolist()
    s["groups"] = [(r * Eh + i if i < Eh else rep_h[r][i - Eh], r * cap + cu_h[r][i],
                    r * cap + cu_h[r][i + 1])
                   for r in range(P) for i in range(NS) if cu_h[r][i + 1] > cu_h[r][i]]
    return E, P * cap


def _rows(n, width, dtype=torch.bfloat16):
    """A buffer for outputs; rows that no slot covers stay as they are."""
    return torch.zeros(n, width, dtype=dtype, device="cuda")


def _prepare_ffn(case, g, s):
    E, M = _prepare_plan(case, g, s)
    h, i = case["hidden"], case["inner"]
    s["x"] = _randn(g, M, h)
    s["w_in"] = _randn(g, E, 2 * i, h, std=h ** -0.5)  # gate rows, then up
    s["w_out"] = _randn(g, E, h, i, std=i ** -0.5)
    s["pre"] = _rows(M, 2 * i) if case["train"] else None
    s["mid"], s["y"] = _rows(M, i), _rows(M, h)


def _prepare_grad(case, g, s):
    E, M = _prepare_plan(case, g, s)
    h, i = case["hidden"], case["inner"]
    s["dy"] = _randn(g, M, h)
    s["w_out"] = _randn(g, E, h, i, std=i ** -0.5)
    if not case["block"]:
        s["mid"] = _randn(g, M, i)
        s["d_mid"] = _rows(M, i, torch.float32)
        s["dw_out"] = torch.empty(E, h, i, device="cuda")
        return
    # what the forward pass kept
    s["x"] = _randn(g, M, h)
    s["w_in"] = _randn(g, E, 2 * i, h, std=h ** -0.5)
    s["pre"] = _randn(g, M, 2 * i)
    s["mid"] = torch.empty(M, i, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, M, 8192):
        gate, up = s["pre"][lo:lo + 8192].float().chunk(2, dim=1)
        s["mid"][lo:lo + 8192] = (gate * torch.sigmoid(gate) * up).bfloat16()
    s["d_pre"], s["dx"] = _rows(M, 2 * i), _rows(M, h)
    s["dw_in"], s["dw_out"] = torch.empty_like(s["w_in"]), torch.empty_like(s["w_out"])


def _prepare_comb(case, g, s):
    t, k, h = case["tokens"], case["k"], case["hidden"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    s["dy"], s["y_exp"] = _randn(g, t, h, dtype=dt), _randn(g, t * k, h, dtype=dt)
    w = torch.rand(t, k, generator=g, device="cuda") + 0.05
    s["w"] = w / w.sum(1, keepdim=True)
    s["pos"] = torch.randperm(t * k, generator=g, device="cuda").int().view(t, k)
    s["dy_exp"] = torch.zeros(t * k, h, dtype=dt, device="cuda")
    s["dw"] = torch.empty(t, k, device="cuda")


def _prepare_lora(case, g, s):
    t, n, k, r, L = case["tokens"], case["n"], case["k"], case["rank"], case["adapters"]
    s["x"] = _randn(g, t, k)
    s["w"] = _randn(g, n, k, std=k ** -0.5)
    s["a"], s["b"] = _randn(g, L, r, k, std=k ** -0.5), _randn(g, L, n, r, std=r ** -0.5)
    s["scale"] = 0.25 + torch.rand(L, generator=g, device="cuda")
    # requests of uneven lengths, one after the other, each with one adapter
    # or (one of six) none
    cut = torch.sort(torch.randperm(t, generator=g, device="cuda")[:case["requests"] - 1])[0]
    at = torch.searchsorted(cut, torch.arange(t, device="cuda"), right=True)
    pick = torch.randint(0, L, (case["requests"],), generator=g, device="cuda")
    none = torch.rand(case["requests"], generator=g, device="cuda") < 1 / 6
    s["adapter"] = torch.where(none, torch.full_like(pick, -1), pick)[at].int()
    s["y"] = torch.empty(t, n, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16,
                         device="cuda")


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"ffn": _own_ffn, "grad": _own_grad, "comb": _own_comb, "lora": _own_lora}[op](s)
    return {"ffn": _plain_ffn, "grad": _plain_grad, "comb": _plain_comb,
            "lora": _plain_lora}[op](s)


# ------------------------------------------------------- through the library

def _kept_plan(mb, s, out):
    c, kept = s["case"], s["kept"]
    if "dims" not in kept:
        P, R, rows = c["ranks"], c["slots"], c["rows"]
        # every pair of the layer is one row of the buffer (top-1 routing has
        # the same layout as top-K over rows / K tokens)
        kept["dims"] = mb.Dims.make(rows, 1, P * c["home"], P, R, c["hidden"], cap=s["cap"],
                                    dtype_in="bf16", dtype_out=out)
        bufs = mb.PlanBuffers.allocate(kept["dims"], s["cu"].device)
        bufs.cu_seqlens, bufs.rep_expert = s["cu"], s["rep"]
        bufs.status.zero_()
        kept["bufs"] = bufs
    return kept["dims"], kept["bufs"]


def _own_ffn(s):
    import token_dispatch_mb_amd as mb

    d, b = _kept_plan(mb, s, "bf16")
    h, i = s["case"]["hidden"], s["case"]["inner"]
    mb.expert_bf16(d, b, i, h, s["x"], s["w_in"], s["mid"], act="swiglu", pre=s["pre"])
    mb.expert_bf16(d, b, h, i, s["mid"], s["w_out"], s["y"])
    return {"y": s["y"], "pre": s["pre"], "mid": s["mid"] if s["case"]["train"] else None}


def _own_grad(s):
    import token_dispatch_mb_amd as mb

    c = s["case"]
    h, i = c["hidden"], c["inner"]
    if not c["block"]:
        d, b = _kept_plan(mb, s, "f32")
        mb.expert_bf16_dgrad(d, b, h, i, s["dy"], s["w_out"], s["d_mid"])
        mb.expert_bf16_wgrad(d, b, h, i, s["dy"], s["mid"], s["dw_out"])
        return {"d_mid": s["d_mid"], "dw_out": s["dw_out"]}
    d, b = _kept_plan(mb, s, "bf16")
    mb.expert_bf16_dgrad(d, b, h, i, s["dy"], s["w_out"], s["d_pre"], act="swiglu", pre=s["pre"])
    mb.expert_bf16_wgrad(d, b, h, i, s["dy"], s["mid"], s["dw_out"])
    mb.expert_bf16_dgrad(d, b, 2 * i, h, s["d_pre"], s["w_in"], s["dx"])
    mb.expert_bf16_wgrad(d, b, 2 * i, h, s["d_pre"], s["x"], s["dw_in"])
    return {"dx": s["dx"], "dw_in": s["dw_in"], "dw_out": s["dw_out"]}


def _own_comb(s):
    import token_dispatch_mb_amd as mb

    c, kept = s["case"], s["kept"]
    if "dims" not in kept:
        t, k = c["tokens"], c["k"]
        # one rank's region holds every pair
        kept["dims"] = mb.Dims.make(t, k, k, 1, 0, c["hidden"], cap=t * k, dtype_in=c["dtype"],
                                    dtype_out=c["dtype"])
        bufs = mb.PlanBuffers.allocate(kept["dims"], s["pos"].device)
        bufs.pos = s["pos"]
        bufs.status.zero_()
        kept["bufs"] = bufs
    mb.combine_grad(kept["dims"], kept["bufs"], s["dy"], s["y_exp"], s["w"], s["dy_exp"], s["dw"])
    return {"dy_exp": s["dy_exp"], "dw": s["dw"]}


def _own_lora(s):
    import token_dispatch_mb_amd as mb

    c, kept = s["case"], s["kept"]
    if "prm" not in kept:
        kept["prm"] = mb.LoraParams.make(c["tokens"], c["n"], c["k"], c["rank"], c["adapters"],
                                         dtype_out=c["out"])
        kept["ws"] = mb.alloc_lora_workspace(kept["prm"], s["x"].device)
    mb.project_lora(kept["prm"], s["x"], s["w"], s["a"], s["b"], s["scale"], s["adapter"],
                    kept["ws"], s["y"])
    return s["y"]


# ------------------------------------------------------------ the plain form

def _plain_ffn(s):
    c = s["case"]
    i = c["inner"]
    for e, lo, hi in s["groups"]:  # ragged groups: two matrix products for each
        pre = s["x"][lo:hi].float() @ s["w_in"][e].float().t()
        gate, up = pre[:, :i], pre[:, i:]
        mid = gate / (1 + torch.exp(-gate)) * up
        s["y"][lo:hi] = (mid @ s["w_out"][e].float().t()).bfloat16()
        if c["train"]:
            s["pre"][lo:hi], s["mid"][lo:hi] = pre.bfloat16(), mid.bfloat16()
    return {"y": s["y"], "pre": s["pre"], "mid": s["mid"] if c["train"] else None}


def _plain_grad(s):
    c = s["case"]
    i = c["inner"]
    if not c["block"]:
        s["dw_out"].zero_()
        for e, lo, hi in s["groups"]:
            dy = s["dy"][lo:hi].float()
            s["d_mid"][lo:hi] = dy @ s["w_out"][e].float()
            s["dw_out"][e] += dy.t() @ s["mid"][lo:hi].float()
        return {"d_mid": s["d_mid"], "dw_out": s["dw_out"]}
    s["dw_in"].zero_()
    s["dw_out"].zero_()
    rest = {}
    for e, lo, hi in s["groups"]:
        rest.setdefault(e, []).append((lo, hi))
    for e, runs in rest.items():  # an expert's replicas add up before the rounding
        w_in, w_out = s["w_in"][e].float(), s["w_out"][e].float()
        dw_in, dw_out = torch.zeros_like(w_in), torch.zeros_like(w_out)
        for lo, hi in runs:
            dy = s["dy"][lo:hi].float()
            gate, up = s["pre"][lo:hi].float().chunk(2, dim=1)
            d_mid = dy @ w_out
            sig = 1 / (1 + torch.exp(-gate))
            d_pre = torch.cat((d_mid * up * sig * (1 + gate * (1 - sig)), d_mid * gate * sig), 1)
            s["dx"][lo:hi] = (d_pre @ w_in).bfloat16()
            dw_in += d_pre.t() @ s["x"][lo:hi].float()
            dw_out += dy.t() @ s["mid"][lo:hi].float()
        s["dw_in"][e], s["dw_out"][e] = dw_in.bfloat16(), dw_out.bfloat16()
    return {"dx": s["dx"], "dw_in": s["dw_in"], "dw_out": s["dw_out"]}


def _plain_comb(s):
    dy = s["dy"].float()
    for j in range(s["case"]["k"]):
        at = s["pos"][:, j].long()
        s["dy_exp"][at] = (s["w"][:, j:j + 1] * dy).to(s["dy_exp"].dtype)
        s["dw"][:, j] = (s["y_exp"][at].float() * dy).sum(1)
    return {"dy_exp": s["dy_exp"], "dw": s["dw"]}


def _plain_lora(s):
    x = s["x"].float()
    y = x @ s["w"].float().t()
    for j in range(s["case"]["adapters"]):
        at = (s["adapter"] == j).nonzero()[:, 0]
        low = (x[at] @ s["a"][j].float().t()) * s["scale"][j]
        y[at] += low @ s["b"][j].float().t()
    return y.to(s["y"].dtype)


# --------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"ffn": _exact_ffn, "grad": _exact_grad, "comb": _exact_comb,
            "lora": _exact_lora}[case["op"]](s)


def _f64(t):
    return t.to(torch.float64)


def _exact_ffn(s):
    c = s["case"]
    M, i, h = s["x"].shape[0], c["inner"], c["hidden"]
    y = torch.zeros(M, h, dtype=torch.float64, device="cuda")
    pre = torch.zeros(M, 2 * i, dtype=torch.float64, device="cuda") if c["train"] else None
    mid = torch.zeros(M, i, dtype=torch.float64, device="cuda") if c["train"] else None
    for e, lo, hi in s["groups"]:
        x = _f64(s["x"][lo:hi])
        gate = torch.mm(x, _f64(s["w_in"][e, :i]).t())
        up = torch.mm(x, _f64(s["w_in"][e, i:]).t())
        act = torch.nn.functional.silu(gate) * up
        torch.mm(act, _f64(s["w_out"][e]).t(), out=y[lo:hi])
        if c["train"]:
            pre[lo:hi, :i], pre[lo:hi, i:], mid[lo:hi] = gate, up, act
    return {"y": y, "pre": pre, "mid": mid}


def _exact_grad(s):
    c = s["case"]
    M, i, h = s["dy"].shape[0], c["inner"], c["hidden"]
    if not c["block"]:
        d_mid = torch.zeros(M, i, dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["dw_out"].shape, dtype=torch.float64, device="cuda")
        for e, lo, hi in s["groups"]:
            dy = _f64(s["dy"][lo:hi])
            torch.mm(dy, _f64(s["w_out"][e]), out=d_mid[lo:hi])
            dw[e].addmm_(dy.t(), _f64(s["mid"][lo:hi]))
        return {"d_mid": d_mid, "dw_out": dw}
    dx = torch.zeros(M, h, dtype=torch.float64, device="cuda")
    dw_in = torch.zeros(s["w_in"].shape, dtype=torch.float64, device="cuda")
    dw_out = torch.zeros(s["w_out"].shape, dtype=torch.float64, device="cuda")
    for e, lo, hi in s["groups"]:
        # the activation's derivatives by automatic differentiation
        pre = _f64(s["pre"][lo:hi]).requires_grad_(True)
        act = torch.nn.functional.silu(pre[:, :i]) * pre[:, i:]
        dy = _f64(s["dy"][lo:hi])
        d_pre, = torch.autograd.grad(act, pre, torch.mm(dy, _f64(s["w_out"][e])))
        dx[lo:hi] = torch.mm(d_pre, _f64(s["w_in"][e]))
        dw_in[e].addmm_(d_pre.t(), _f64(s["x"][lo:hi]))
        dw_out[e].addmm_(dy.t(), _f64(s["mid"][lo:hi]))
    return {"dx": dx, "dw_in": dw_in, "dw_out": dw_out}


def _exact_comb(s):
    dy, at = _f64(s["dy"]), s["pos"].long()
    rows = torch.zeros(s["y_exp"].shape, dtype=torch.float64, device="cuda")
    rows[at.view(-1)] = (_f64(s["w"])[:, :, None] * dy[:, None, :]).view(-1, dy.shape[1])
    dw = torch.stack([torch.linalg.vecdot(_f64(s["y_exp"][at[:, j]]), dy)
                      for j in range(at.shape[1])], 1)
    return {"dy_exp": rows, "dw": dw}


def _exact_lora(s):
    x = _f64(s["x"])
    y = torch.mm(x, _f64(s["w"]).t())
    for j in torch.unique(s["adapter"]).tolist():
        if j >= 0:
            rows = s["adapter"] == j
            low = torch.mm(x[rows], _f64(s["a"][j]).t())
            y[rows] += float(s["scale"][j]) * torch.mm(low, _f64(s["b"][j]).t())
    return y
