"""Cases of the operators around an MoE layer's dispatch and combine: norm, experts' products, routing gradients.

Each case describes one pass of one operator as a training or serving step calls it:

* ``norm``: the residual stream takes up a layer's output, its RMS norm goes to the router and, in 8 bits with
  block scales, to the dispatch; ``norm_grad`` is its backward pass.
* ``product``: the grouped rows that a dispatch delivers times their experts' weights, with bias, activation and
  residual in the epilogue; without top-k every rank has one dense product. ``product_grad`` is its backward pass.
* ``route_grad``: the backward passes of combine and dispatch.

With ``own`` false, ``run`` computes the pass from elementary torch operations; with ``own`` true it calls
the library. ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
BLOCK = 128   # values that share a scale


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _norm(name, rows, hidden, dtype, residual, quant):
    return dict(name=name, op="norm", rows=rows, hidden=hidden, dtype=dtype, residual=residual, quant=quant)


def _norm_grad(name, rows, hidden, dtype, residual):
    return dict(name=name, op="norm_grad", rows=rows, hidden=hidden, dtype=dtype, residual=residual)


def _product(name, ranks, tokens, experts, topk, k, n, act, dtype="bf16", bias=False, residual=False, pre=False,
             skew=False):
    return dict(name=name, op="product", ranks=ranks, tokens=tokens, experts=experts, topk=topk, k=k, n=n, act=act,
                dtype=dtype, bias=bias, residual=residual, pre=pre, skew=skew)


def _product_grad(name, ranks, tokens, experts, topk, k, n, act, bias, skew=False):
    return dict(name=name, op="product_grad", ranks=ranks, tokens=tokens, experts=experts, topk=topk, k=k, n=n,
                act=act, bias=bias, skew=skew)


def _route_grad(name, ranks, tokens, experts, topk, hidden, add, skew=False):
    return dict(name=name, op="route_grad", ranks=ranks, tokens=tokens, experts=experts, topk=topk, hidden=hidden,
                add=add, skew=skew)


def listed():
    return [
        # One decoded token: launch latency.
        _norm("norm_token", 1, 7168, "bf16", True, True),
        # The prefill workload's 8 x 4096 tokens on their way into the router and a block-fp8 dispatch.
        _norm("norm_prefill", 32768, 7168, "bf16", True, True),
        # Its backward pass; the residual stream brings a gradient of its own.
        _norm_grad("norm_train", 32768, 7168, "bf16", True),
        # The smallest workload, pre-activations kept for training: launch latency.
        _product("product_tiny", 4, 16, 16, 2, 256, 512, "swiglu", bias=True, pre=True),
        # One decoded token on one rank: eight experts' weights are read for a row each.
        _product("product_token", 1, 1, 64, 8, 7168, 2048, "swiglu"),
        # The decode workload: 256 experts of about 128 rows each.
        _product("product_decode", 32, 128, 256, 8, 7168, 2048, "swiglu"),
        # The prefill workload on the codes and block scales that a block-fp8 dispatch delivers.
        _product("product_prefill_fp8", 8, 4096, 256, 8, 7168, 2048, "swiglu", dtype="fp8"),
        # The down product of an expert that sees every token, added to what the others give.
        _product("product_shared", 1, 4096, 1, 0, 2048, 7168, "none", residual=True),
        # Ragged rows of odd sizes, one of the experts popular: gradients of a small layer.
        _product_grad("product_grad_small", 1, 333, 6, 2, 520, 264, "gelu", bias=True, skew=True),
        # A training step's up product: rows, weights and bias.
        _product_grad("product_grad", 8, 1024, 64, 8, 7168, 2048, "swiglu", bias=True),
        # Gradients of combine and dispatch at the decode workload's size.
        _route_grad("route_grad_decode", 32, 128, 256, 8, 7168, False),
        # The same at the prefill workload's size, added to the gradient that comes past the experts.
        _route_grad("route_grad_prefill", 8, 4096, 256, 8, 7168, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _routing(rng, most_slots):
    """Ranks, tokens per rank, experts, top-k and whether few experts are popular."""
    ranks = rng.choice([1, 1, 2, 4, 8, 32])
    experts = ranks * _log(rng, 1, 256 // ranks)
    topk = min(experts, rng.choice([1, 2, 4, 6, 8, 8, 9]))
    tokens = _log(rng, 1, max(1, min(4096, most_slots // (ranks * topk))))
    return ranks, tokens, experts, topk, rng.random() < 0.4


def draw(rng: random.Random):
    op = rng.choice(["norm", "norm", "norm_grad", "product", "product", "product", "product_grad", "product_grad",
                     "route_grad", "route_grad"])
    if op in ("norm", "norm_grad"):
        quant = op == "norm" and rng.random() < 0.6
        hidden = BLOCK * _log(rng, 1, 64) if quant else 8 * _log(rng, 1, 1024)
        rows = _log(rng, 1, min(65536, 32768 * 7168 // hidden))
        dtype, residual = rng.choice(["bf16", "bf16", "fp16"]), rng.random() < 0.7
        case = _norm("", rows, hidden, dtype, residual, quant) if op == "norm" else \
            _norm_grad("", rows, hidden, dtype, residual)
    elif op == "route_grad":
        ranks, tokens, experts, topk, skew = _routing(rng, 262144)
        case = _route_grad("", ranks, tokens, experts, topk, 8 * _log(rng, 16, 896), rng.random() < 0.5, skew)
    else:
        fp8 = op == "product" and rng.random() < 0.35
        unit = BLOCK if fp8 else 8
        k, n = unit * _log(rng, max(1, 64 // unit), 7168 // unit), unit * _log(rng, max(1, 64 // unit), 7168 // unit)
        act = rng.choice(["none", "silu", "gelu", "swiglu", "swiglu"])
        ranks, tokens, experts, topk, skew = _routing(rng, 65536)
        if rng.random() < 0.25:   # dense
            ranks = experts = rng.choice([1, 1, 2])
            tokens, topk, skew = _log(rng, 1, 16384 // ranks), 0, False
        while experts * k * n > 1 << 30:
            n = max(unit, n // 2 // unit * unit)
            k = max(unit, k * 2 // 3 // unit * unit)
        bias = rng.random() < 0.5
        if op == "product":
            case = _product("", ranks, tokens, experts, topk, k, n, act, "fp8" if fp8 else "bf16", bias,
                            rng.random() < 0.4, not fp8 and rng.random() < 0.4, skew)
        else:
            case = _product_grad("", ranks, tokens, experts, topk, k, n, act, bias, skew)
        while work(case)["flops"] > 7e12:
            case["tokens"] //= 2
    return {key: v for key, v in case.items() if key != "name"}


def _weight_rows(c):
    return 2 * c["n"] if c["act"] == "swiglu" else c["n"]


def _slots(c):
    return c["ranks"] * c["tokens"] * max(1, c["topk"])


def _cap(c):
    """Rows of each rank's grouped buffer: all of them on one rank, else a quarter more than the mean."""
    mean = c["tokens"] * max(1, c["topk"])
    if c["ranks"] == 1 or c["topk"] == 0:
        return mean
    return min(mean + mean // 4 + 64, c["ranks"] * c["tokens"] * max(c["topk"], c["experts"] // c["ranks"]))


def _experts_used(c):
    """Experts that meet a row, on average, when all are equally popular."""
    if c["topk"] == 0:
        return c["experts"]
    return c["experts"] * (1 - (1 - c["topk"] / c["experts"]) ** (c["ranks"] * c["tokens"]))


def work(case):
    c, op = case, case["op"]
    if op == "norm":
        per = 2 + 2 + (4 if c["residual"] else 0) + (1 + 4 / BLOCK if c["quant"] else 0)
        return {"bytes": c["rows"] * c["hidden"] * per + 2 * c["hidden"], "flops": 6 * c["rows"] * c["hidden"]}
    if op == "norm_grad":
        per = 2 * (4 if c["residual"] else 3)
        return {"bytes": c["rows"] * c["hidden"] * per + 6 * c["hidden"], "flops": 10 * c["rows"] * c["hidden"]}
    rows = _slots(c)
    if op == "route_grad":
        tokens, h = c["ranks"] * c["tokens"], c["hidden"]
        # The expert rows, their gradients out and in; dout, dx and what is added; weights, their gradients, the plan.
        return {"bytes": 3 * 2 * rows * h + (3 if c["add"] else 2) * 2 * tokens * h + 16 * rows,
                "flops": 4 * rows * h + (1 + c["topk"]) * tokens * h}
    wrows, used = _weight_rows(c), _experts_used(c)
    weights = used * wrows * c["k"]
    flops = 2 * rows * wrows * c["k"]
    if op == "product":
        es, scale = (1, 1) if c["dtype"] == "fp8" else (2, 0)
        total = es * weights + scale * 4 * weights / BLOCK ** 2 + rows * c["k"] * (es + scale * 4 / BLOCK)
        total += rows * 2 * (c["n"] * (2 if c["residual"] else 1) + (wrows if c["pre"] else 0))
        return {"bytes": total + (2 * used * wrows if c["bias"] else 0), "flops": flops}
    # Rows and their gradient, dout and the pre-activations; weights read, all their gradients written.
    pre = wrows if c["act"] != "none" else 0
    total = rows * 2 * (2 * c["k"] + c["n"] + pre) + 2 * weights + 2 * c["experts"] * wrows * c["k"]
    return {"bytes": total + (4 * c["experts"] * wrows if c["bias"] else 0), "flops": 2 * flops}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(shape, g, dtype=torch.bfloat16, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)
    return x if scale == 1.0 else x.mul_(scale)


def _empty(shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _zeros(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def _prepare_norm(c, seed):
    g, shape, dtype = _gen(seed), (c["rows"], c["hidden"]), DTYPES[c["dtype"]]
    s = {"case": c, "x": _randn(shape, g, dtype), "weight": 1 + 0.1 * _randn(c["hidden"], g, dtype),
         "residual": _randn(shape, g, dtype, 3.0) if c["residual"] else None}
    if c["op"] == "norm":
        s["sum"] = _empty(shape, dtype) if c["residual"] else None
        s["y"] = _empty(shape, dtype)
        s["codes"] = _empty(shape, torch.float8_e4m3fn) if c["quant"] else None
        s["scales"] = _empty((c["rows"], c["hidden"] // BLOCK), torch.float32) if c["quant"] else None
    else:
        s["dy"] = _randn(shape, g, dtype)
        s["dx"], s["dweight"] = _empty(shape, dtype), _empty(c["hidden"], torch.float32)
    if own:
        import combine_ep_plan_amd as ep
        s["ep"] = ep
        if c["op"] == "norm_grad":
            s["ws"] = _empty(ep.rms_norm_grad_bytes(c["rows"], c["hidden"]), torch.uint8)
    return s


def _route(s, c, g):
    """Expert ids of every slot and, from them, each slot's row in the grouped buffers (N * cap: dropped) and each
    expert's first row and number of rows."""
    n, t, e, k, cap = c["ranks"], c["tokens"], c["experts"], c["topk"], _cap(c)
    local = e // n
    if k == 0:
        s["groups"] = [(d * cap, cap) for d in range(n)]
        return
    score = torch.rand((n * t, e), device=DEV, generator=g).log_().neg_().log_().neg_()
    if c["skew"]:   # Zipf 1.2
        popular = torch.randperm(e, device=DEV, generator=g).float().add_(1).log_().mul_(-1.2)
        score += popular
    s["idx"] = score.topk(k, 1)[1].to(torch.int32).view(n, t, k)
    flat = s["idx"].flatten().long()
    count = torch.zeros(e, dtype=torch.long, device=DEV).index_add_(0, flat, torch.ones_like(flat))
    end = count.view(n, local).cumsum(1)
    first = (end - count.view(n, local)).flatten()   # in the rank's buffer
    order = torch.sort(flat, stable=True)[1]
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=DEV) - (count.cumsum(0) - count)[flat[order]]
    row = first[flat] + place
    s["rows"] = torch.where(row < cap, flat // local * cap + row, n * cap).view(n * t, k)
    lo, hi = first.clamp(max=cap), end.flatten().clamp(max=cap)
    s["groups"] = [(i // local * cap + a, b - a) for i, (a, b) in enumerate(zip(lo.tolist(), hi.tolist()))]


def _plan(s, c, hidden, payload=None):
    """The library's descriptor and, for routed rows, its plan."""
    import combine_ep_plan_amd as ep
    s["ep"] = ep
    s["desc"] = ep.make_desc(c["ranks"], c["tokens"], hidden, c["experts"], max(1, c["topk"]),
                             ep.EP_PAYLOAD_BF16 if payload is None else payload, _cap(c))
    s["plan"] = None
    if c["topk"]:
        s["plan"] = _empty(ep.plan_bytes(s["desc"]), torch.uint8)
        ep.plan(s["desc"], s["idx"], s["plan"], _zeros(1, torch.int32))


def _fp8(shape, g):
    """Codes of a bell curve that uses most of the type's range."""
    x = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    for part in (x.view(-1, *shape[1:]) if len(shape) > 2 else [x]):
        part.copy_(torch.randn(part.shape, device=DEV, generator=g).mul_(100).clamp_(-448, 448))
    return x


def _prepare_product(c, seed):
    g = _gen(seed)
    s = {"case": c}
    _route(s, c, g)
    rows, wrows, e, k, n = c["ranks"] * _cap(c), _weight_rows(c), c["experts"], c["k"], c["n"]
    if c.get("dtype") == "fp8":
        s["x"] = [_fp8((rows, k), g), (torch.rand((rows, k // BLOCK), device=DEV, generator=g) + 0.5) / 100]
        s["w"] = _fp8((e, wrows, k), g)
        s["w_scale"] = (torch.rand((e, wrows // BLOCK, k // BLOCK), device=DEV, generator=g) + 0.5) / (100 * k ** 0.5)
    else:
        s["x"] = [_randn((rows, k), g)]
        s["w"], s["w_scale"] = _randn((e, wrows, k), g, scale=k ** -0.5), None
    s["bias"] = _randn((e, wrows), g) if c["bias"] else None
    if c["op"] == "product":
        s["residual"] = _randn((rows, n), g) if c["residual"] else None
        s["pre"] = _zeros((rows, wrows)) if c["pre"] else None
        s["out"] = _zeros((rows, n))
    else:
        s["dout"] = _randn((rows, n), g)
        s["pre"] = _randn((rows, wrows), g) if c["act"] != "none" else None
        s["dx"], s["dw"] = _zeros((rows, k)), _empty((e, wrows, k))
        s["dbias"] = _empty((e, wrows), torch.float32) if c["bias"] else None
    if own:
        import combine_ep_plan_amd as ep
        _plan(s, c, k, ep.EP_PAYLOAD_FP8_B128 if c.get("dtype") == "fp8" else None)
        act = {"none": ep.EP_ACT_NONE, "silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU, "swiglu": ep.EP_ACT_SWIGLU}
        s["product"] = ep.make_product(s["w"], act[c["act"]], w_scale=s["w_scale"], bias=s["bias"])
        if c["op"] == "product_grad":
            s["ws"] = _empty(ep.expert_product_grad_bytes(s["desc"], s["product"]), torch.uint8)
    return s


def _prepare_route_grad(c, seed):
    g = _gen(seed)
    s = {"case": c}
    _route(s, c, g)
    n, t, h, k, cap = c["ranks"], c["tokens"], c["hidden"], c["topk"], _cap(c)
    s["dout"], s["y"] = _randn((n, t, h), g), _randn((n * cap, h), g)
    s["dgrouped"] = _randn((n * cap, h), g)
    s["weights"] = torch.softmax(torch.randn((n, t, k), device=DEV, generator=g), -1)
    s["add"] = _randn((n, t, h), g) if c["add"] else None
    # One row more than the library's: dropped slots of the plain form go there.
    s["dy"], s["dweights"], s["dx"] = _zeros((n * cap + 1, h)), _empty((n, t, k), torch.float32), _empty((n, t, h))
    if own:
        _plan(s, c, h)
    return s


def prepare(case, seed):
    if case["op"] in ("norm", "norm_grad"):
        return _prepare_norm(case, seed)
    if case["op"] == "route_grad":
        return _prepare_route_grad(case, seed)
    return _prepare_product(case, seed)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        s["sum"].copy_(h + s["residual"].float())
        h = s["sum"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    s["y"].copy_(y)
    if s["codes"] is not None:
        blocks = y.view(y.shape[0], -1, BLOCK)
        top = blocks.abs().amax(-1)
        scale = torch.where(top > 0, top / 448, torch.ones_like(top))
        s["scales"].copy_(scale)
        s["codes"].copy_((blocks / scale[..., None]).clamp(-448, 448).view_as(y))


def _plain_norm_grad(s):
    """`x` holds the normed rows, `residual` the gradient that arrives on the residual stream."""
    h, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    unit = h * rstd
    g = dy * w
    dx = rstd * (g - unit * (g * unit).mean(1, keepdim=True))
    s["dx"].copy_(dx if s["residual"] is None else dx + s["residual"].float())
    s["dweight"].copy_((dy * unit).sum(0))


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "swiglu":
        gate, up = z.chunk(2, -1)
        return gate * torch.sigmoid(gate) * up
    return z


def _act_grad(z, d, act):
    if act in ("silu", "swiglu"):
        gate, up = z.chunk(2, -1) if act == "swiglu" else (z, None)
        sig = torch.sigmoid(gate)
        slope = sig * (1 + gate * (1 - sig))
        return d * slope if up is None else torch.cat([d * up * slope, d * gate * sig], -1)
    if act == "gelu":
        return d * (0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5)
    return d


def _wide(x, scale, rows, to):
    """Rows, or an expert's weights, as numbers of type `to`; scale blocks hold 128 columns and `rows` rows."""
    if scale is None:
        return x.to(to)
    return x.to(to) * scale.to(to).repeat_interleave(rows, 0).repeat_interleave(BLOCK, 1)


def _plain_product(s):
    c = s["case"]
    for e, (at, n) in enumerate(s["groups"]):
        if n == 0:
            continue
        r = slice(at, at + n)
        x = _wide(s["x"][0][r], s["x"][1][r] if len(s["x"]) > 1 else None, 1, torch.float32)
        w = _wide(s["w"][e], None if s["w_scale"] is None else s["w_scale"][e], BLOCK, torch.float32)
        z = x @ w.t()
        if s["bias"] is not None:
            z += s["bias"][e].float()
        if s["pre"] is not None:
            s["pre"][r] = z.to(torch.bfloat16)
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"][r].float()
        s["out"][r] = y.to(torch.bfloat16)


def _plain_product_grad(s):
    for e, (at, n) in enumerate(s["groups"]):
        r = slice(at, at + n)
        dz = s["dout"][r].float()
        if s["pre"] is not None:
            dz = _act_grad(s["pre"][r].float(), dz, s["case"]["act"])
        if s["dbias"] is not None:
            s["dbias"][e] = dz.sum(0)
        if n == 0:
            s["dw"][e] = 0
            continue
        s["dx"][r] = (dz @ s["w"][e].float()).to(torch.bfloat16)
        s["dw"][e] = (dz.t() @ s["x"][0][r].float()).to(torch.bfloat16)


def _plain_route_grad(s):
    c = s["case"]
    h, k = c["hidden"], c["topk"]
    dout, w, last = s["dout"].view(-1, h).float(), s["weights"].view(-1, k), s["dy"].shape[0] - 1
    dx = torch.zeros_like(dout) if s["add"] is None else s["add"].view(-1, h).float()
    for i in range(k):
        row = s["rows"][:, i]
        here = (row < last)[:, None]
        at = row.clamp(max=last - 1)
        s["dweights"].view(-1, k)[:, i] = (torch.where(here, s["y"][at].float(), 0) * dout).sum(1)
        s["dy"][row] = (w[:, i, None] * dout).to(torch.bfloat16)
        dx = dx + torch.where(here, s["dgrouped"][at].float(), 0)
    s["dy"][last] = 0
    s["dx"].copy_(dx.view_as(s["dx"]))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_norm(s):
    if own:
        s["ep"].rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], sum=s["sum"], y=s["y"], codes=s["codes"],
                         scales=s["scales"])
    else:
        _plain_norm(s)
    return {name: s[name] for name in ("sum", "y", "codes", "scales") if s[name] is not None}


def _run_norm_grad(s):
    if own:
        s["ep"].rms_norm_grad(s["dy"], s["x"], s["weight"], EPS, s["dx"], s["dweight"], s["ws"], dsum=s["residual"])
    else:
        _plain_norm_grad(s)
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _run_product(s):
    if own:
        s["ep"].expert_product(s["desc"], s["product"], s["x"], s["plan"], s["out"], residual=s["residual"],
                               pre=s["pre"])
    else:
        _plain_product(s)
    return {name: s[name] for name in ("out", "pre") if s[name] is not None}


def _run_product_grad(s):
    if own:
        s["ep"].expert_product_grad(s["desc"], s["product"], s["dout"], s["x"][0], s["pre"], s["plan"], s["ws"],
                                    dx=s["dx"], dw=s["dw"], dbias=s["dbias"])
    else:
        _plain_product_grad(s)
    return {name: s[name] for name in ("dx", "dw", "dbias") if s[name] is not None}


def _run_route_grad(s):
    if own:
        s["ep"].combine_grad(s["desc"], s["dout"], s["y"], s["weights"], s["plan"], s["dy"], s["dweights"])
        s["ep"].dispatch_grad(s["desc"], s["dgrouped"], s["plan"], s["dx"], add=s["add"])
    else:
        _plain_route_grad(s)
    return {"dy": s["dy"], "dweights": s["dweights"], "dx": s["dx"]}


def run(state):
    return {"norm": _run_norm, "norm_grad": _run_norm_grad, "product": _run_product,
            "product_grad": _run_product_grad, "route_grad": _run_route_grad}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _chunks(rows, width):
    step = max(1, (1 << 28) // width)
    return [slice(a, min(rows, a + step)) for a in range(0, rows, step)]


def _exact_norm(s):
    c = s["case"]
    shape = (c["rows"], c["hidden"])
    out = {"y": _empty(shape, torch.float64)}
    if s["residual"] is not None:
        out["sum"] = _empty(shape, torch.float64)
    if c["quant"]:
        out["codes"], out["scales"] = _empty(shape, torch.float32), _empty(s["scales"].shape, torch.float64)
    for r in _chunks(*shape):
        h = s["x"][r].double()
        if s["residual"] is not None:
            out["sum"][r] = h + s["residual"][r].double()
            h = out["sum"][r].to(s["x"].dtype).double()   # the stream holds the rounded sum
        y = h * s["weight"].double() / (torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / c["hidden"]
                                        + EPS).sqrt()
        out["y"][r] = y
        if c["quant"]:
            scale = y.unflatten(1, (-1, BLOCK)).abs().max(-1).values / 448
            scale[scale == 0] = 1
            out["scales"][r] = scale
            out["codes"][r] = (y / torch.repeat_interleave(scale, BLOCK, 1)).clamp(-448, 448).float()
    return out


def _exact_norm_grad(s):
    c = s["case"]
    dx = _empty((c["rows"], c["hidden"]), torch.float64)
    dweight = _zeros(c["hidden"], torch.float64)
    for r in _chunks(c["rows"], c["hidden"]):
        h, dy, w = s["x"][r].double(), s["dy"][r].double(), s["weight"].double()
        var = (h * h).sum(1, keepdim=True) / c["hidden"] + EPS
        dot = (dy * w * h).sum(1, keepdim=True) / c["hidden"]
        dx[r] = (dy * w * var - h * dot) / var ** 1.5
        if s["residual"] is not None:
            dx[r] += s["residual"][r].double()
        dweight += (dy * h / var.sqrt()).sum(0)
    return {"dx": dx, "dweight": dweight}


def _exact_product(s):
    c, n = s["case"], s["case"]["n"]
    out = {"out": _zeros(s["out"].shape, torch.float64)}
    if s["pre"] is not None:
        out["pre"] = _zeros(s["pre"].shape, torch.float64)
    for e in range(c["experts"]):
        at, m = s["groups"][e]
        if not m:
            continue
        x, w = s["x"][0][at:at + m].double(), s["w"][e].double()
        if s["w_scale"] is not None:
            x = (x.unflatten(1, (-1, BLOCK)) * s["x"][1][at:at + m].double()[..., None]).flatten(1)
            blocks = w.view(w.shape[0] // BLOCK, BLOCK, -1, BLOCK)
            w = (blocks * s["w_scale"][e].double()[:, None, :, None]).view_as(w)
        z = torch.mm(x, w.T)
        z = z if s["bias"] is None else z + s["bias"][e].double()
        if s["pre"] is not None:
            out["pre"][at:at + m] = z
        if c["act"] == "swiglu":
            y = z[:, :n] / (1 + torch.exp(-z[:, :n])) * z[:, n:]
        elif c["act"] == "silu":
            y = z / (1 + torch.exp(-z))
        elif c["act"] == "gelu":
            y = z * torch.special.ndtr(z)
        else:
            y = z
        out["out"][at:at + m] = y if s["residual"] is None else y + s["residual"][at:at + m].double()
    return out


def _exact_product_grad(s):
    c, n = s["case"], s["case"]["n"]
    out = {"dx": _zeros(s["dx"].shape, torch.float64), "dw": _zeros(s["dw"].shape, torch.float64)}
    if s["dbias"] is not None:
        out["dbias"] = _zeros(s["dbias"].shape, torch.float64)
    for e in range(c["experts"]):
        at, m = s["groups"][e]
        if not m:
            continue
        d, x, w = s["dout"][at:at + m].double(), s["x"][0][at:at + m].double(), s["w"][e].double()
        if c["act"] != "none":
            z = s["pre"][at:at + m].double()
            gate = z[:, :n]
            sig = 1 / (1 + torch.exp(-gate))
            if c["act"] == "gelu":
                d = d * (torch.special.ndtr(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi))
            elif c["act"] == "silu":
                d = d * (sig + gate * sig * (1 - sig))
            else:
                d = torch.cat([d * z[:, n:] * (sig + gate * sig * (1 - sig)), d * gate * sig], 1)
        out["dx"][at:at + m] = torch.mm(d, w)
        out["dw"][e] = torch.mm(d.T, x)
        if s["dbias"] is not None:
            out["dbias"][e] = d.sum(0)
    return out


def _exact_route_grad(s):
    c, h, last = s["case"], s["case"]["hidden"], s["dy"].shape[0] - 1
    tokens = c["ranks"] * c["tokens"]
    out = {"dy": _zeros(s["dy"].shape, torch.float64), "dweights": _zeros(s["dweights"].shape, torch.float64),
           "dx": _zeros(s["dx"].shape, torch.float64)}
    dout, w = s["dout"].view(tokens, h), s["weights"].view(tokens, -1)
    dw, dx = out["dweights"].view(tokens, -1), out["dx"].view(tokens, h)
    if s["add"] is not None:
        dx += s["add"].view(tokens, h)
    for r in _chunks(tokens, h * c["topk"]):
        row, d = s["rows"][r], dout[r].double()
        slot = (row < last).nonzero()   # token within the chunk, choice
        token, choice = slot[:, 0], slot[:, 1]
        at = row[token, choice]
        out["dy"][at] = w[r].double()[token, choice][:, None] * d[token]
        dw[r][token, choice] = (s["y"][at].double() * d[token]).sum(1)
        dx[r].index_add_(0, token, s["dgrouped"][at].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "product": _exact_product,
            "product_grad": _exact_product_grad, "route_grad": _exact_route_grad}[case["op"]](s)
