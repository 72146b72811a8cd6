"""Cases and plain forms of the operators around the routed experts: the norm in front
of the router, the routing of given logits, the gradient of the combine, and the dense
linear layer, forward and backward.

``run`` computes a case in elementary torch operations (32 bits; 64 where the choice of
experts depends on values next to one another), or, with ``own`` set, by the library's
entry points on the same state. ``exact`` gives the definitions in 64 bits.
"""
import functools
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
SCALE = 2.5  # routed scaling factor of the route cases


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one serving step of 128 sequences: the norm of the hidden states before the router
        norm("norm_decode", "forward", "layer", "bf16", 128, 7168),
        # the prefill batch of the 896-expert layer; statistics kept for the backward pass
        norm("norm_prefill", "forward", "layer", "bf16", 16384, 7168),
        # a training step's gradient of the same norm, weight and bias gradients included
        norm("norm_train", "backward", "layer", "bf16", 8192, 7168),
        # routing of one serving step: 384 experts, top 8, balance bias
        route("route_decode", "forward", "f32", 128, 384, 8, 1, 1, "sigmoid", True, True, 0.0),
        # prefill, group-limited 4 of 8 groups; a batch padded to its longest sequence
        route("route_prefill", "forward", "f32", 8192, 384, 8, 8, 4, "sigmoid", True, True, 0.1),
        # training with 896 fine-grained experts, bf16 logits from a mixed-precision router,
        # softmax over all experts without renormalisation: every logit has a gradient
        route("route_train", "backward", "bf16", 16384, 896, 16, 1, 1, "softmax", False, False, 0.0),
        # training: gradients of expert rows and routing weights, 4096 tokens, top 8
        combine("combine_train", 4096, 7168, 8, 0.0),
        # a small fine-tuning batch, some pairs dropped by the router (padding)
        combine("combine_small", 96, 7168, 6, 0.05),
        # one token through a projection (serving one sequence)
        linear("linear_token", "forward", "bf16", 1, 2048, 7168, "silu", True, False, False),
        # prefill of a dense layer's output projection with its residual
        linear("linear_prefill", "forward", "bf16", 8192, 7168, 2048, "none", True, True, False),
        # a ragged batch in fp16, sizes that fill no tile, pre-activation kept for training
        linear("linear_ragged", "forward", "f16", 1037, 2051, 1111, "gelu", True, True, True),
        # a training step of a dense layer's first projection
        linear("linear_train", "backward", "bf16", 4096, 2048, 7168, "silu", True, False, True),
    ]


def norm(name, way, kind, dtype, T, H):
    return {"name": name, "op": "norm", "way": way, "kind": kind, "dtype": dtype, "T": T, "H": H}


def route(name, way, dtype, T, E, k, groups, kept, score, renorm, bias, padded):
    return {"name": name, "op": "route", "way": way, "dtype": dtype, "T": T, "E": E, "k": k,
            "groups": groups, "kept": kept, "score": score, "renorm": renorm, "bias": bias,
            "padded": padded}


def combine(name, T, H, k, dropped):
    return {"name": name, "op": "combine", "way": "backward", "T": T, "H": H, "k": k,
            "dropped": dropped}


def linear(name, way, dtype, M, N, K, act, bias, residual, pre):
    return {"name": name, "op": "linear", "way": way, "dtype": dtype, "M": M, "N": N, "K": K,
            "act": act, "bias": bias, "residual": residual, "pre": pre}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "combine", "linear"])
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        H = rng.choice([_log(rng, 8, 16384), 8 * _log(rng, 16, 2048)])
        T = _log(rng, 1, min(16384, 16384 * 7168 * 2 // (H * SIZE[dtype])))
        c = norm("", rng.choice(["forward", "backward"]), rng.choice(["layer", "rms"]), dtype, T, H)
    elif op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * max(2, _log(rng, 16, 1024) // groups)
        kept = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(16, kept * (E // groups)))
        c = route("", rng.choice(["forward", "forward", "backward"]), rng.choice(["f32", "bf16", "f16"]),
                  _log(rng, 1, 16384), E, k, groups, kept,
                  rng.choice(["sigmoid", "softmax", "sqrtsoftplus"]), rng.random() < 0.7,
                  rng.random() < 0.7, rng.choice([0.0, 0.2]))
    elif op == "combine":
        k = rng.randint(1, 16)
        H = 128 * rng.randint(1, 64)
        c = combine("", _log(rng, 1, min(8192, 4096 * 8 * 7168 // (k * H))), H, k,
                    rng.choice([0.0, 0.1]))
    else:
        N, K = _log(rng, 16, 8192), _log(rng, 16, 8192)
        M = _log(rng, 1, min(8192, 8192 * 2048 * 7168 // (3 * N * K)))
        way = rng.choice(["forward", "forward", "backward"])
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
        c = linear("", way, rng.choice(["bf16", "f16"]), M, N, K, act, rng.random() < 0.7,
                   way == "forward" and rng.random() < 0.5,
                   act != "none" if way == "backward" else rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------------------- inputs
def _rows(g, rows, cols, dtype, scale=1.0):
    """A matrix whose rows start on 16-byte boundaries, as a program pads odd widths."""
    ld = -(-cols // 8) * 8
    t = torch.randn(rows, ld, generator=g, device="cuda") * scale
    return t.to(dtype)[:, :cols]


def _out(rows, cols, dtype):
    return torch.empty(rows, -(-cols // 8) * 8, dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = functools.partial(torch.randn, generator=g, device="cuda")
    s = {"case": case}
    i32 = dict(dtype=torch.int32, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    if case["op"] == "norm":
        T, H, dt = case["T"], case["H"], TYPES[case["dtype"]]
        # hidden states of a residual stream: rows of unlike size, a little off centre
        s["x"] = ((rand(T, H) + 0.1) * torch.exp(0.5 * rand(T, 1))).to(dt)
        s["w"] = 1.0 + 0.2 * rand(H)
        s["b"] = 0.1 * rand(H) if case["kind"] == "layer" else None
        s["eps"] = 1e-6
        s["mean"] = torch.empty(T, **f32) if case["kind"] == "layer" else None
        s["rstd"] = torch.empty(T, **f32)
        s["y"] = torch.empty(T, H, dtype=dt, device="cuda")
        if case["way"] == "backward":
            xf = s["x"].float()
            mean = xf.mean(1) if case["kind"] == "layer" else torch.zeros(T, **f32)
            s["rstd"] = 1.0 / torch.sqrt((xf - mean[:, None]).square().mean(1) + s["eps"])
            s["mean"] = mean if case["kind"] == "layer" else None
            s["dy"] = rand(T, H).to(dt)
            s["dw"] = torch.empty(H, **f32)
            s["db"] = torch.empty(H, **f32) if case["kind"] == "layer" else None
    elif case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # logits of a router of std 0.02 over 7168 normalised features
        l = 1.7 * rand(T, E)
        pad = torch.rand(T, generator=g, device="cuda") < case["padded"]
        if case["way"] == "forward":
            l = l.masked_fill(pad[:, None], -math.inf)  # padded tokens choose nothing
        s["logits"] = l.to(TYPES[case["dtype"]])
        s["bias"] = 0.2 * torch.rand(E, generator=g, device="cuda") - 0.1 if case["bias"] else None
        s["idx"] = torch.empty(T, k, **i32)
        s["w"] = torch.empty(T, k, **f32)
        if case["way"] == "backward":
            order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)[1]
            s["idx"] = order[:, :k].masked_fill(pad[:, None], -1).to(torch.int32).contiguous()
            s["dw"] = rand(T, k)
            s["dlogits"] = torch.empty_like(s["logits"])
    elif case["op"] == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        N = T * k
        s["y"] = (0.5 * rand(N, H)).bfloat16()
        s["dout"] = rand(T, H).bfloat16()
        s["w"] = torch.rand(T, k, generator=g, device="cuda") * 0.5
        # every pair's row in expert order; dropped pairs have none
        row_of = torch.argsort(torch.rand(N, generator=g, device="cuda")).to(torch.int32)
        s["row_of"] = row_of.masked_fill(
            torch.rand(N, generator=g, device="cuda") < case["dropped"], -1)
        s["dy"] = torch.zeros(N, H, dtype=torch.bfloat16, device="cuda")
        s["dw"] = torch.empty(T, k, **f32)
    else:
        M, N, K, dt = case["M"], case["N"], case["K"], TYPES[case["dtype"]]
        s["x"] = _rows(g, M, K, dt)
        s["w"] = _rows(g, N, K, dt, K ** -0.5)
        s["bias"] = 0.1 * rand(N) if case["bias"] else None
        s["residual"] = _rows(g, M, N, dt) if case["residual"] else None
        s["y"] = _out(M, N, dt)
        s["pre"] = _out(M, N, dt) if case["pre"] else None
        if case["way"] == "backward":
            s["dy"] = _rows(g, M, N, dt)
            if case["pre"]:
                s["pre"] = _rows(g, M, N, dt)
            s["dx"], s["dw"] = _out(M, K, dt), _out(N, K, dt)
            s["db"] = torch.empty(N, **f32) if case["bias"] else None
    return s


# ------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    forms = _OWN if own else _PLAIN
    return forms[case["op"], case["way"]](state, case)


def _norm_forward(s, c):
    x = s["x"].float()
    mean = x.sum(1) / c["H"] if c["kind"] == "layer" else None
    d = x - mean[:, None] if mean is not None else x
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / c["H"] + s["eps"])
    y = d * rstd[:, None] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_backward(s, c):
    dy, x, rstd = s["dy"].float(), s["x"].float(), s["rstd"][:, None]
    layer = c["kind"] == "layer"
    xh = (x - s["mean"][:, None] if layer else x) * rstd
    g = dy * s["w"]
    dx = g - xh * ((g * xh).sum(1, keepdim=True) / c["H"])
    if layer:
        dx = dx - g.sum(1, keepdim=True) / c["H"]
    return {"dx": (dx * rstd).to(s["x"].dtype), "dw": (dy * xh).sum(0),
            "db": dy.sum(0) if layer else None}


def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    if score == "sqrtsoftplus":
        return torch.sqrt(torch.clamp(l, min=0) + torch.log1p(torch.exp(-l.abs())))
    top = l.max(1, keepdim=True)[0]
    e = torch.exp(l - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    z = e.sum(1, keepdim=True)
    return e / torch.where(z > 0, z, torch.ones_like(z))


def _route_forward(s, c):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double() + 0.0
    score = _scores(l, c["score"])
    sel = score + s["bias"].double() if s["bias"] is not None else score
    sel = sel.masked_fill(torch.isinf(l), -math.inf)
    if G > 1:
        by = sel.view(T, G, E // G)
        first, at = by.max(2, keepdim=True)
        second = by.scatter(2, at, -math.inf).max(2)[0]
        gscore = torch.where(torch.isinf(second), first[:, :, 0], first[:, :, 0] + second)
        order = torch.sort(gscore, dim=1, descending=True, stable=True)[1][:, :c["kept"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        sel = sel.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    # the larger s + bias first, then the larger logit, then the lower index
    by_logit = torch.sort(l, dim=1, descending=True, stable=True)[1]
    got, order = torch.sort(sel.gather(1, by_logit), dim=1, descending=True, stable=True)
    idx = by_logit.gather(1, order)[:, :k]
    none = torch.isinf(got[:, :k])
    w = score.gather(1, idx).masked_fill(none, 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return {"idx": idx.masked_fill(none, -1).to(torch.int32), "w": (w * SCALE).float()}



def _route_backward(s, c):
    l = s["logits"].float()
    none = s["idx"] < 0
    idx = s["idx"].clamp(min=0).long()
    score = _scores(l, c["score"])
    p = score.gather(1, idx).masked_fill(none, 0.0)
    g = s["dw"].masked_fill(none, 0.0) * SCALE
    if c["renorm"]:
        total = p.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        g = (g - (g * p).sum(1, keepdim=True) / total) / total
    g = g.masked_fill(none, 0.0)
    if c["score"] == "softmax":
        ds = torch.zeros_like(l).scatter_add_(1, idx, g)
        dl = score * (ds - (g * p).sum(1, keepdim=True))
    else:
        lk = l.gather(1, idx)
        sig = 1.0 / (1.0 + torch.exp(-lk))
        slope = p * (1.0 / (1.0 + torch.exp(lk))) if c["score"] == "sigmoid" else \
            0.5 * sig / torch.where(none, torch.ones_like(p), p)
        dl = torch.zeros_like(l).scatter_add_(1, idx, g * slope)
    return {"dlogits": dl.to(s["logits"].dtype)}


def _combine_backward(s, c):
    T, H, k = c["T"], c["H"], c["k"]
    rows = s["row_of"].long()
    none = rows < 0
    dout = s["dout"].float()
    pair = torch.arange(T * k, device=rows.device)
    pair_of = torch.full((T * k + 1,), -1, device=rows.device)
    pair_of[rows.masked_fill(none, T * k)] = pair
    pair_of = pair_of[:T * k]
    at = pair_of.clamp(min=0)
    dy = (dout[at // k] * s["w"].view(-1)[at][:, None]).bfloat16()
    s["dy"].copy_(torch.where((pair_of < 0)[:, None], s["dy"], dy))  # rows of no pair stay
    dots = (dout[pair // k] * s["y"][rows.clamp(min=0)].float()).sum(1)
    return {"dy": s["dy"], "dw": dots.masked_fill(none, 0.0).view(T, k)}


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return sig * (1.0 + z * (1.0 - sig))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi)
    t = torch.tanh(u * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * u * (1.0 + 3 * 0.044715 * z * z)


def _linear_forward(s, c):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    dt = s["x"].dtype
    return {"y": y.to(dt), "pre": z.to(dt) if c["pre"] else None}


def _linear_backward(s, c):
    g = s["dy"].float()
    if c["act"] != "none":
        g = g * _slope(s["pre"].float(), c["act"])
    dt = s["x"].dtype
    return {"dx": (g @ s["w"].float()).to(dt), "dw": (g.t() @ s["x"].float()).to(dt),
            "db": g.sum(0) if c["bias"] else None}


_PLAIN = {("norm", "forward"): _norm_forward, ("norm", "backward"): _norm_backward,
          ("route", "forward"): _route_forward, ("route", "backward"): _route_backward,
          ("combine", "backward"): _combine_backward,
          ("linear", "forward"): _linear_forward, ("linear", "backward"): _linear_backward}


# ------------------------------------------------------------- the library's entry points
def _moe():
    import expert_routing_grouped_layer_b200 as moe
    return moe


@functools.lru_cache(maxsize=64)
def _config(hidden, E, k, groups, kept, score, renorm):
    """The layer configuration a program holds for its router and combine."""
    from expert_routing_grouped_layer_b200 import workloads
    moe = _moe()
    return moe.make_config(workloads.CONFIGS["tiny_bf16"].replace(
        hidden=hidden, n_routed_experts=E, num_experts_per_tok=k, n_group=groups, topk_group=kept,
        score_fn=score, norm_topk_prob=renorm, routed_scaling_factor=SCALE))


def _workspace(s, nbytes):
    """The program's workspace, made once."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_norm_forward(s, c):
    _moe().moe_norm(s["x"], s["w"], s["b"], s["eps"], s["y"], s["mean"], s["rstd"], kind=c["kind"])
    return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}


def _own_norm_backward(s, c):
    moe = _moe()
    ws = _workspace(s, moe.moe_norm_backward_workspace_bytes(c["T"], c["H"]))
    moe.moe_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["y"], s["dw"], s["db"],
                          ws, kind=c["kind"])
    return {"dx": s["y"], "dw": s["dw"], "db": s["db"]}


def _own_route_forward(s, c):
    cfg = _config(128, c["E"], c["k"], c["groups"], c["kept"], c["score"], c["renorm"])
    _moe().moe_route(cfg, s["logits"], s["bias"], s["idx"], s["w"])
    return {"idx": s["idx"], "w": s["w"]}


def _own_route_backward(s, c):
    cfg = _config(128, c["E"], c["k"], c["groups"], c["kept"], c["score"], c["renorm"])
    _moe().moe_route_backward(cfg, s["logits"], s["idx"], s["dw"], s["dlogits"])
    return {"dlogits": s["dlogits"]}


def _own_combine_backward(s, c):
    cfg = _config(c["H"], 64, c["k"], 1, 1, "sigmoid", True)
    _moe().moe_combine_backward(cfg, s["dout"], s["y"], s["row_of"], s["w"], s["dy"], s["dw"])
    return {"dy": s["dy"], "dw": s["dw"]}


def _own_linear_forward(s, c):
    _moe().moe_linear(s["x"], s["w"], s["bias"], s["residual"], s["y"], s["pre"], act=c["act"])
    return {"y": s["y"], "pre": s["pre"]}


def _own_linear_backward(s, c):
    moe = _moe()
    ws = _workspace(s, moe.moe_linear_backward_workspace_bytes(c["M"], c["N"], c["K"], c["act"]))
    moe.moe_linear_backward(s["dy"], s["x"], s["w"], s["pre"], s["dx"], s["dw"], s["db"], ws,
                            act=c["act"])
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


_OWN = {("norm", "forward"): _own_norm_forward, ("norm", "backward"): _own_norm_backward,
        ("route", "forward"): _own_route_forward, ("route", "backward"): _own_route_backward,
        ("combine", "backward"): _own_combine_backward,
        ("linear", "forward"): _own_linear_forward, ("linear", "backward"): _own_linear_backward}


# ------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "norm":
        n, e = c["T"] * c["H"], SIZE[c["dtype"]]
        layer = c["kind"] == "layer"
        if c["way"] == "forward":
            return {"bytes": 2 * n * e + 4 * c["H"] * (1 + layer) + 4 * c["T"] * (1 + layer),
                    "flops": 8 * n}
        return {"bytes": 3 * n * e + 4 * c["H"] * (2 + layer) + 4 * c["T"] * (1 + layer),
                "flops": 14 * n}
    if c["op"] == "route":
        n, e = c["T"] * c["E"], SIZE[c["dtype"]]
        if c["way"] == "forward":
            return {"bytes": n * e + 8 * c["T"] * c["k"] + (4 * c["E"] if c["bias"] else 0),
                    "flops": 10 * n}
        # the gradient of every logit; the logits themselves where a softmax needs them all,
        # else those of the chosen experts
        dense = c["score"] == "softmax" and not c["renorm"]
        read = n * e if dense else c["T"] * c["k"] * e
        return {"bytes": n * e + read + 8 * c["T"] * c["k"], "flops": 6 * n}
    if c["op"] == "combine":
        pairs = c["T"] * c["k"] * (1 - c["dropped"])
        return {"bytes": 2 * c["H"] * (c["T"] + 2 * pairs) + 12 * c["T"] * c["k"],
                "flops": 3 * pairs * c["H"]}
    M, N, K = c["M"], c["N"], c["K"]
    if c["way"] == "forward":
        return {"bytes": 2 * (M * K + N * K + M * N * (1 + c["residual"] + c["pre"]))
                + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    return {"bytes": 2 * (2 * M * K + 2 * N * K + M * N * (1 + c["pre"]))
            + (4 * N if c["bias"] else 0), "flops": 4 * M * N * K}


# ------------------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"], case["way"]](s, case)


def _exact_norm_forward(s, c):
    x = s["x"].double()
    if c["kind"] == "layer":
        var, mean = torch.var_mean(x, dim=1, correction=0)
    else:
        var, mean = x.square().mean(1), None
    scale = torch.rsqrt(var + float(s["eps"]))
    y = torch.empty_like(x)
    torch.sub(x, mean[:, None] if mean is not None else 0.0, out=y)
    y.mul_(scale[:, None]).mul_(s["w"].double())
    return {"y": y.add_(s["b"].double()) if s["b"] is not None else y, "mean": mean, "rstd": scale}


def _exact_norm_backward(s, c):
    # y_h = w_h n_h + b_h with n = (x - mean) r: dn = w dy, then the part of dn along n (and,
    # for the layer norm, along the ones) is taken out
    n = s["x"].double()
    if c["kind"] == "layer":
        n = n - s["mean"].double()[:, None]
    n = n * s["rstd"].double()[:, None]
    dy = s["dy"].double()
    dn = dy * s["w"].double()
    along = torch.einsum("th,th->t", dn, n) / c["H"]
    dx = dn - n * along[:, None]
    if c["kind"] == "layer":
        dx -= dn.mean(1, keepdim=True)
    return {"dx": dx * s["rstd"].double()[:, None], "dw": torch.einsum("th,th->h", dy, n),
            "db": dy.sum(0) if c["kind"] == "layer" else None}


def _exact_scores(l, score):
    if score == "sigmoid":
        return torch.special.expit(l)
    if score == "sqrtsoftplus":
        return torch.logaddexp(l, torch.zeros_like(l)).sqrt()
    return torch.softmax(l, 1).nan_to_num(0.0)


def _exact_route_forward(s, c):
    # experts one after another: the best of what is left, k times
    T, E, G = c["T"], c["E"], c["groups"]
    l = s["logits"].double()
    score = _exact_scores(l, c["score"])
    left = score if s["bias"] is None else score + s["bias"].double()
    left = left.masked_fill(l == -math.inf, -math.inf)
    if G > 1:
        two = left.view(T, G, -1).topk(2, dim=2)[0]
        value = two[..., 0] + two[..., 1].masked_fill(two[..., 1] == -math.inf, 0.0)
        open_ = torch.zeros_like(value, dtype=torch.bool)
        for _ in range(c["kept"]):
            at = value.argmax(1, keepdim=True)
            open_.scatter_(1, at, True)
            value = value.scatter(1, at, -math.inf)
        left = torch.where(open_[:, :, None].expand(T, G, E // G).reshape(T, E), left,
                           torch.full_like(left, -math.inf))
    idx, w = [], []
    for _ in range(c["k"]):
        best, at = left.max(1, keepdim=True)
        empty = best == -math.inf
        w.append(torch.where(empty, torch.zeros_like(best), score.gather(1, at)))
        idx.append(torch.where(empty, torch.full_like(at, -1), at))
        left = left.scatter(1, at, -math.inf)
    w = torch.cat(w, 1)
    if c["renorm"]:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    return {"idx": torch.cat(idx, 1).to(torch.int32), "w": w * SCALE}


def _exact_route_backward(s, c):
    # by differentiating the forward definition at the chosen experts
    l = s["logits"].double().requires_grad_(True)
    has = s["idx"] >= 0
    p = _exact_scores(l, c["score"]).gather(1, s["idx"].clamp(min=0).long())
    p = torch.where(has, p, torch.zeros_like(p))
    if c["renorm"]:
        total = p.sum(1, keepdim=True)
        p = p / torch.where(has.any(1, keepdim=True), total, torch.ones_like(total))
    loss = (torch.where(has, s["dw"].double(), torch.zeros_like(p)) * p * SCALE).sum()
    return {"dlogits": torch.autograd.grad(loss, l)[0]}


def _exact_combine_backward(s, c):
    T, H, k = c["T"], c["H"], c["k"]
    rows = s["row_of"].view(T, k).long()
    dy = s["dy"].double()
    dw = torch.zeros(T, k, dtype=torch.float64, device=dy.device)
    for j in range(k):
        has = (rows[:, j] >= 0).nonzero()[:, 0]
        at = rows[has, j]
        g = s["dout"][has].double()
        dy[at] = g * s["w"][has, j].double()[:, None]
        dw[has, j] = torch.einsum("th,th->t", g, s["y"][at].double())
    return {"dy": dy, "dw": dw}


def _exact_linear_forward(s, c):
    bias = s["bias"].double() if s["bias"] is not None else None
    z = torch.nn.functional.linear(s["x"].double(), s["w"].double(), bias)
    f = torch.nn.functional
    y = {"none": lambda v: v, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
         "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[c["act"]](z)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y, "pre": z if c["pre"] else None}


def _exact_linear_backward(s, c):
    g = s["dy"].double()
    if c["act"] != "none":
        f = torch.nn.functional
        z = s["pre"].double().requires_grad_(True)
        y = {"relu": f.relu, "silu": f.silu, "gelu": f.gelu,
             "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[c["act"]](z)
        g = torch.autograd.grad(y, z, g)[0]
    return {"dx": torch.einsum("mn,nk->mk", g, s["w"].double()),
            "dw": torch.einsum("mn,mk->nk", g, s["x"].double()),
            "db": g.sum(0) if c["bias"] else None}


_EXACT = {("norm", "forward"): _exact_norm_forward, ("norm", "backward"): _exact_norm_backward,
          ("route", "forward"): _exact_route_forward,
          ("route", "backward"): _exact_route_backward,
          ("combine", "backward"): _exact_combine_backward,
          ("linear", "forward"): _exact_linear_forward,
          ("linear", "backward"): _exact_linear_backward}
