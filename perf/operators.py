"""Measured cases of the operators around plan, dispatch and combine.

Four operators of a mixture-of-experts layer, each in a plain form of
elementary torch operations (``own`` false) and through this library (``own``
true):

* route  — router logits to expert ids and gate weights: softmax or sigmoid
  scores, a balance bias that counts for the choice only, expert groups,
  top-K in descending order (ties to the lowest id), renormalised weights;
* norm   — root-mean-square norm with the residual's addition, rows out in
  fp8 e4m3 with one fp32 scale per 128 elements (what the dispatch takes);
* quant  — rows to microscaled 4-bit floats (e2m1 elements, one e8m0 scale
  per 32) and back;
* expert — the experts' products over the dispatch buffer in that format,
  alone or after the gated activation that quantises its input.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a small batch through an 8-expert layer
        _route("route_small", 50, 8, 2, "f32", "softmax"),
        # a decode layer of 256 experts in 8 groups, balance bias, bf16 logits
        _route("route_decode", 8192, 256, 8, "bf16", "sigmoid", bias=True, groups=8, top_groups=4,
               group_top=2, scale=2.5),
        # the same router over a whole prefill batch, fp32 logits
        _route("route_prefill", 131072, 256, 8, "f32", "sigmoid", bias=True, groups=8,
               top_groups=4, group_top=2, scale=2.5),
        # 384 experts, ungrouped softmax scores, weights renormalised
        _route("route_384", 65536, 384, 8, "f32", "softmax"),
        # one token's row ahead of a decode layer, normed rows kept for the router
        _norm("norm_token", 1, 7168, "bf16", residual=True, rows=True),
        # fp32 rows of an odd count, no residual
        _norm("norm_odd", 4099, 4224, "f32", residual=False, rows=True),
        # a prefill batch: the residual stream updated, fp8 rows for the dispatch
        _norm("norm_prefill", 131072, 7168, "bf16", residual=True, rows=False),
        # a small fp32 weight matrix of odd height, quantised on loading and read back
        _quant("quant_weight", 2501, 1152, "f32"),
        # the token rows of a decode layer, quantised for the dispatch and read back
        _quant("quant_decode", 8192, 7168, "bf16"),
        # a small decode batch: two or three rows for each expert, weights stream through once
        _expert("expert_few", rows=512, ranks=64, home=4, slots=1, n=2048, k=7168, swiglu=False),
        # a decode layer's second product: gated activation, quantisation, product
        _expert("expert_decode_down", rows=65536, ranks=64, home=4, slots=1, n=7168, k=2048,
                swiglu=True),
        # a prefill layer's first product over 32 ranks' full regions
        _expert("expert_prefill", rows=1048576, ranks=32, home=8, slots=1, n=2048, k=7168,
                swiglu=False),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("route", "norm", "quant", "expert"))
    if op == "route":
        experts = rng.choice((8, 16, 48, 60, 64, 100, 128, 160, 256, 320, 384, 512))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0])
        size = experts // groups
        top_groups = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(10, top_groups * size))
        score, bias = rng.choice(("softmax", "sigmoid")), rng.random() < 0.5
        return _route(None, log_int(1, 131072 * 256 // max(experts, 256)), experts, k,
                      rng.choice(("f32", "bf16")), score, bias=bias, groups=groups,
                      top_groups=top_groups, group_top=rng.choice((1, 2)) if size > 1 else 1,
                      renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)))
    if op == "norm":
        return _norm(None, log_int(1, 60000), 128 * log_int(1, 64), rng.choice(("bf16", "f32")),
                     residual=rng.random() < 0.6, rows=rng.random() < 0.5)
    if op == "quant":
        return _quant(None, log_int(1, 50000), 128 * log_int(1, 64), rng.choice(("bf16", "f32")))
    ranks, home = rng.choice(((1, 8), (8, 1), (8, 8), (16, 8), (32, 8), (64, 4)))
    return _expert(None, rows=ranks * log_int(1, 200000 // ranks), ranks=ranks, home=home,
                   slots=rng.choice((0, 1, 2)), n=8 * log_int(8, 512), k=128 * log_int(1, 40),
                   swiglu=rng.random() < 0.4, out=rng.choice(("bf16", "bf16", "f32")))


def _named(name, case):
    return case if name is None else dict(case, name=name)


def _route(name, tokens, experts, k, dtype, score, bias=False, groups=1, top_groups=1,
           group_top=1, renorm=True, scale=1.0):
    return _named(name, dict(op="route", tokens=tokens, experts=experts, k=k, dtype=dtype,
                             score=score, bias=bias, groups=groups, top_groups=top_groups,
                             group_top=group_top, renorm=renorm, scale=scale))


def _norm(name, tokens, hidden, dtype, residual, rows):
    return _named(name, dict(op="norm", tokens=tokens, hidden=hidden, dtype=dtype,
                             residual=residual, rows=rows))


def _quant(name, rows, hidden, dtype):
    return _named(name, dict(op="quant", rows=rows, hidden=hidden, dtype=dtype))


def _expert(name, rows, ranks, home, slots, n, k, swiglu, out="bf16"):
    return _named(name, dict(op="expert", rows=rows, ranks=ranks, home=home, slots=slots, n=n, k=k,
                             swiglu=swiglu, out=out))


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": t * e * _size(case) + t * k * 8 + (4 * e if case["bias"] else 0),
                "flops": 4 * t * e}
    if op == "norm":
        n, b = case["tokens"] * case["hidden"], _size(case)
        ends = 1 + (2 if case["residual"] else 0) + (1 if case["rows"] else 0)
        return {"bytes": n * b * ends + n + n // 32 + case["hidden"] * b, "flops": 6 * n}
    if op == "quant":
        n = case["rows"] * case["hidden"]
        # quantise (read the row, write codes and scales), then read those back into rows
        return {"bytes": 2 * n * _size(case) + 2 * (n // 2 + n // 32), "flops": 4 * n}
    rows, n, k = case["rows"], case["n"], case["k"]
    slots = case["ranks"] * (case["home"] + case["slots"])
    used = slots * (1 - math.exp(-rows / slots))  # slots that get a row at all
    experts = min(case["ranks"] * case["home"], used)
    packed = k // 2 + k // 32
    b_in = rows * (4 * k if case["swiglu"] else packed)
    b_out = 4 if case["out"] == "f32" else 2
    return {"bytes": b_in + experts * n * packed + rows * n * b_out, "flops": 2 * rows * n * k}


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case, "kept": {}}
    {"route": _prepare_route, "norm": _prepare_norm, "quant": _prepare_quant,
     "expert": _prepare_expert}[case["op"]](case, g, s)
    return s


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_route(case, g, s):
    t, e = case["tokens"], case["experts"]
    # noise over a long-tailed popularity, as a trained router's logits are
    rank = torch.argsort(torch.rand(e, generator=g, device="cuda")).float() + 1
    s["logits"] = (_randn(g, t, e) - 0.4 * torch.log(rank)).to(_dtype(case["dtype"]))
    s["bias"] = 0.05 * _randn(g, e) if case["bias"] else None
    s["ids"] = torch.empty(t, case["k"], dtype=torch.int32, device="cuda")
    s["w"] = torch.empty(t, case["k"], device="cuda")


def _prepare_norm(case, g, s):
    t, h, dt = case["tokens"], case["hidden"], _dtype(case["dtype"])
    s["x"] = _randn(g, t, h).to(dt)
    s["residual"] = (4 * _randn(g, t, h)).to(dt) if case["residual"] else None
    s["weight"] = (1 + 0.1 * _randn(g, h)).to(dt)
    s["eps"] = 1e-6
    s["residual_out"] = torch.empty(t, h, dtype=dt, device="cuda") if case["residual"] else None
    s["y"] = torch.empty(t, h, dtype=dt, device="cuda") if case["rows"] else None
    s["q"] = torch.empty(t, h, dtype=torch.uint8, device="cuda")
    s["q_scale"] = torch.empty(t, h // 128, device="cuda")


def _prepare_quant(case, g, s):
    m, h, dt = case["rows"], case["hidden"], _dtype(case["dtype"])
    # each row at a level of its own, as activations and weight rows are
    s["x"] = (_randn(g, m, h) * torch.exp(_randn(g, m, 1))).to(dt)
    s["q"] = torch.empty(m, h // 2, dtype=torch.uint8, device="cuda")
    s["q_scale"] = torch.empty(m, h // 32, dtype=torch.uint8, device="cuda")
    s["back"] = torch.empty(m, h, dtype=dt, device="cuda")


def _codes(g, m, h, level):
    """Rows in 4 bits and their scales, as a quantiser leaves them: random
    elements, scales within a few powers of two of `level`."""
    q = torch.randint(0, 256, (m, h // 2), generator=g, device="cuda", dtype=torch.uint8)
    sc = torch.randint(level - 2, level + 2, (m, h // 32), generator=g, device="cuda",
                       dtype=torch.uint8)
    return q, sc


def _prepare_expert(case, g, s):
    P, Eh, R, rows, n, k = (case["ranks"], case["home"], case["slots"], case["rows"], case["n"],
                            case["k"])
    E, NS, cap = P * Eh, Eh + R, rows // P  # a balanced plan: every rank serves its full region
    # the plan of the layer: replicas of experts homed elsewhere, some slots
    # empty, rows skewed over the slots of a rank
    rep = torch.randint(0, E, (P, max(R, 1)), generator=g, device="cuda", dtype=torch.int32)
    at = torch.arange(P, device="cuda", dtype=torch.int32)[:, None]
    drop = (rep // Eh == at) | (torch.rand(rep.shape, generator=g, device="cuda") < 0.2)
    rep = torch.where(drop, torch.full_like(rep, -1), rep)
    share = torch.rand((P, NS), generator=g, device="cuda") ** 2 + 0.05
    if R:
        share[:, Eh:] = torch.where(rep < 0, torch.zeros_like(share[:, Eh:]), share[:, Eh:])
    cdf = torch.cumsum(share, 1)
    cdf = cdf / cdf[:, -1:]
    u = torch.rand((P, cap), generator=g, device="cuda")
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
    s["b"], s["b_scale"] = _codes(g, E * n, k, 121)
    if case["swiglu"]:
        s["x"] = _randn(g, P * cap, 2 * k).to(torch.bfloat16)
        s["a"] = torch.empty(P * cap, k // 2, dtype=torch.uint8, device="cuda")
        s["a_scale"] = torch.empty(P * cap, k // 32, dtype=torch.uint8, device="cuda")
        s["row_src"] = torch.zeros(P * cap, dtype=torch.int32, device="cuda")
    else:
        s["a"], s["a_scale"] = _codes(g, P * cap, k, 126)
    s["out"] = torch.zeros(P * cap, n, dtype=_dtype(case["out"]), device="cuda")


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"route": _own_route, "norm": _own_norm, "quant": _own_quant,
                "expert": _own_expert}[op](s)
    return {"route": _plain_route, "norm": _plain_norm, "quant": _plain_quant,
            "expert": _plain_expert}[op](s)


# ------------------------------------------------------- through the library

def _own_route(s):
    import token_dispatch_mb_amd as mb

    c, kept = s["case"], s["kept"]
    if "prm" not in kept:
        kept["prm"] = mb.RouteParams.make(
            c["tokens"], c["experts"], c["k"], dtype=c["dtype"], score=c["score"],
            n_groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
            renorm=c["renorm"], scale=c["scale"])
    mb.route(kept["prm"], s["logits"], s["ids"], s["w"], bias=s["bias"])
    return {"ids": s["ids"], "w": s["w"]}


def _own_norm(s):
    import token_dispatch_mb_amd as mb

    mb.rmsnorm_fp8(s["x"], s["weight"], s["eps"], s["q"], s["q_scale"], residual=s["residual"],
                   residual_out=s["residual_out"], y=s["y"])
    return {"q": s["q"].view(torch.float8_e4m3fn), "q_scale": s["q_scale"],
            "residual": s["residual_out"], "y": s["y"]}


def _own_quant(s):
    import token_dispatch_mb_amd as mb

    mb.quantize_mx4(s["x"], s["q"], s["q_scale"])
    mb.dequantize_mx4(s["q"], s["q_scale"], s["back"])
    return s["back"]


def _own_expert(s):
    import token_dispatch_mb_amd as mb

    c, kept = s["case"], s["kept"]
    if "dims" not in kept:
        P, R, rows = c["ranks"], c["slots"], c["rows"]
        # every pair of the layer is one row of the buffer (top-1 routing has
        # the same layout as top-K over rows / K tokens)
        kept["dims"] = mb.Dims.make(rows, 1, P * c["home"], P, R, c["n"], cap=s["cap"],
                                    dtype_in="bf16", dtype_out=c["out"])
        bufs = mb.PlanBuffers.allocate(kept["dims"], s["cu"].device)
        bufs.cu_seqlens, bufs.rep_expert = s["cu"], s["rep"]
        bufs.status.zero_()
        kept["bufs"] = bufs
    if c["swiglu"]:
        mb.quantize_mx4(s["x"], s["a"], s["a_scale"], act="swiglu", row_src=s["row_src"])
    mb.expert_mx4(kept["dims"], kept["bufs"], c["n"], c["k"], s["a"], s["a_scale"], s["b"],
                  s["b_scale"], s["out"])
    return s["out"]


# ------------------------------------------------------------ the plain form

def _plain_route(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["k"]
    # 64 bits: which expert is chosen turns on the smallest difference of scores
    l = s["logits"].double()
    if c["score"] == "softmax":
        x = torch.exp(l - l.amax(1, keepdim=True))
        score = x / x.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-l))
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        by = choice.view(t, c["groups"], e // c["groups"])
        best = torch.sort(by, dim=2, descending=True)[0][:, :, : c["group_top"]].sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True)[1][:, : c["top_groups"]]
        open_ = torch.zeros_like(best).scatter_(1, keep, 1.0) > 0
        choice = torch.where(open_[:, :, None], by, torch.full_like(by, -math.inf)).view(t, e)
    ids = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.int(), "w": (w * c["scale"]).float()}


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    out = h.to(s["x"].dtype) if s["residual"] is not None else None
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    by = y.view(y.shape[0], -1, 128)
    amax = by.abs().amax(2)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (by / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view_as(y).to(torch.float8_e4m3fn)
    return {"q": q, "q_scale": scale, "residual": out,
            "y": y.to(s["x"].dtype) if s["y"] is not None else None}


def _to_mx4(x):
    """float32 rows rounded to microscaled 4-bit values (as float32)."""
    by = x.view(x.shape[0], -1, 32)
    amax = by.abs().amax(2, keepdim=True)
    # 2^(floor(log2 amax) - 2): the block's largest value lands in [4, 8)
    e = torch.clamp(torch.frexp(amax)[1] - 3, -126, 127)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    unit = ((e + 127) << 23).view(torch.float32)
    v = by / unit
    a = v.abs()
    r = torch.where(a < 2, torch.round(2 * a) / 2,
                    torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2))).clamp(max=6)
    return (torch.copysign(r, v) * unit).view_as(x)


def _from_codes(q, sc, table):
    """float32 rows of packed 4-bit codes (low nibble first) and e8m0 scales."""
    v = torch.stack((table[(q & 15).int()], table[(q >> 4).int()]), dim=-1)
    unit = (sc.int() << 23).view(torch.float32)
    return (v.view(q.shape[0], -1, 32) * unit[:, :, None]).view(q.shape[0], -1)


def _table():
    return torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")


def _plain_quant(s):
    return _to_mx4(s["x"].float()).to(s["x"].dtype)


def _plain_expert(s):
    c, out, table = s["case"], s["out"], _table()
    n = c["n"]
    for e, lo, hi in s["groups"]:  # ragged groups: one matrix product for each
        if c["swiglu"]:
            gate, up = s["x"][lo:hi].float().chunk(2, dim=1)
            a = _to_mx4(gate / (1 + torch.exp(-gate)) * up)
        else:
            a = _from_codes(s["a"][lo:hi], s["a_scale"][lo:hi], table)
        b = _from_codes(s["b"][e * n:(e + 1) * n], s["b_scale"][e * n:(e + 1) * n], table)
        out[lo:hi] = (a @ b.t()).to(out.dtype)
    return out


# --------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "quant": _exact_quant,
            "expert": _exact_expert}[case["op"]](s)


def _exact_route(s):
    # the ids have no rounding; the weights follow from the chosen logits
    c = s["case"]
    l = s["logits"].to(torch.float64)
    if c["score"] == "sigmoid":
        score = torch.where(l >= 0, 1 / (1 + torch.exp(-l.abs())),
                            torch.exp(-l.abs()) / (1 + torch.exp(-l.abs())))
    else:
        score = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    choice = score.clone() if s["bias"] is None else score + s["bias"].to(torch.float64)
    size = c["experts"] // c["groups"]
    if c["groups"] > 1:
        rest = choice.view(-1, c["groups"], size).clone()
        total = torch.zeros(rest.shape[:2], dtype=torch.float64, device=rest.device)
        for _ in range(c["group_top"]):
            best, at = rest.max(2, keepdim=True)
            total += best[:, :, 0]
            rest.scatter_(2, at, -math.inf)
        limit = total.kthvalue(c["groups"] - c["top_groups"] + 1, dim=1, keepdim=True)[0]
        closed = (total < limit).repeat_interleave(size, dim=1)
        choice.masked_fill_(closed, -math.inf)
    picked = []
    for _ in range(c["k"]):
        at = choice.argmax(1, keepdim=True)
        picked.append(score.gather(1, at))
        choice.scatter_(1, at, -math.inf)
    w = torch.cat(picked, 1)
    if c["renorm"]:
        w /= w.sum(1, keepdim=True)
    return {"ids": None, "w": w * c["scale"]}


def _exact_norm(s):
    h = s["x"].to(torch.float64)
    if s["residual"] is not None:
        h += s["residual"].to(torch.float64)
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / h.shape[1] + s["eps"])
    y *= s["weight"].to(torch.float64)
    # the rows before their rounding to 8 bits
    blocks = y.reshape(y.shape[0], -1, 128)
    scale = torch.linalg.vector_norm(blocks, math.inf, dim=2) / E4M3_MAX
    scale[scale == 0] = 1
    q = (blocks / scale.unsqueeze(2)).reshape(y.shape)
    return {"q": q, "q_scale": scale, "residual": h if s["residual"] is not None else None,
            "y": y if s["y"] is not None else None}


def _exact_mx4(x):
    """float64 rows at the nearest microscaled 4-bit values, ties to the even
    code: found among the midpoints of the element's eight magnitudes."""
    by = x.reshape(x.shape[0], -1, 32)
    top = by.abs().max(2, keepdim=True)[0]
    level = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    level = torch.where(torch.exp2(level) > top, level - 1, level)  # log2 rounded up
    level = torch.where(2 * torch.exp2(level) <= top, level + 1, level)
    unit = torch.exp2(level - 2)
    mag = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mids = (mag[1:] + mag[:-1]) / 2
    a = (by / unit).abs().contiguous()
    low, high = torch.searchsorted(mids, a, right=False), torch.searchsorted(mids, a, right=True)
    code = torch.where(low == high, low, torch.where(low % 2 == 0, low, high))
    return (mag[code] * torch.sign(by) * unit).reshape(x.shape)


def _exact_quant(s):
    x = s["x"]
    step = max(1, (1 << 26) // x.shape[1])
    return torch.cat([_exact_mx4(x[i:i + step].to(torch.float64))
                      for i in range(0, x.shape[0], step)])


def _exact_expert(s):
    c = s["case"]
    n, k = c["n"], c["k"]
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def rows_of(q, sc):
        nib = torch.empty(q.shape[0], k, dtype=torch.int64, device="cuda")
        nib[:, 0::2], nib[:, 1::2] = q % 16, q // 16
        v = mag[nib % 8] * (1 - 2 * (nib // 8))
        return v * torch.exp2(sc.to(torch.float64) - 127).repeat_interleave(32, dim=1)

    y = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e, lo, hi in s["groups"]:
        w = rows_of(s["b"][e * n:(e + 1) * n], s["b_scale"][e * n:(e + 1) * n])
        if c["swiglu"]:
            x = s["x"][lo:hi].to(torch.float64)
            a = _exact_mx4(x[:, :k] * torch.sigmoid(x[:, :k]) * x[:, k:])
        else:
            a = rows_of(s["a"][lo:hi], s["a_scale"][lo:hi])
        torch.mm(a, w.t(), out=y[lo:hi])
    return y
