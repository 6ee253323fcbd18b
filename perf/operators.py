"""Cases of the mixture-of-experts sublayer's operators: layer norm, routing, the experts' products, combine.

The sublayer produces the expert gradients [experts, fan_out, fan_in] that the Newton–Schulz library
orthogonalizes.  A case names an operator ("op"), a pass ("fwd": the forward pass alone, as in serving; "bwd": the
gradients from a saved forward pass; "step": forward and gradients, as in training), its sizes and its type.

`run` computes a case in elementary torch operations where `own` is false, and with the library's entry points where
it is true; `exact` is the operators' definition in 64 bits.
"""

import math

import torch

own = False

EPS = 1e-5     # layer norm
TINY = 1e-20   # added to the sum of the chosen scores before they are renormalised

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one token's norm in serving: latency
        {"name": "norm_token", "op": "norm", "pass": "fwd", "rows": 1, "cols": 2048, "dtype": "bf16", "params": "bf16"},
        # rows that no vector width divides, everything in fp32
        {"name": "norm_odd", "op": "norm", "pass": "step", "rows": 1003, "cols": 1531, "dtype": "fp32",
         "params": "fp32"},
        # a training batch at the widest hidden size, fp32 master parameters
        {"name": "norm_train", "op": "norm", "pass": "step", "rows": 8192, "cols": 7168, "dtype": "bf16",
         "params": "fp32"},
        # one token choosing among 128 experts: latency
        {"name": "route_token", "op": "route", "pass": "fwd", "tokens": 1, "experts": 128, "top_k": 8, "groups": 1,
         "top_groups": 1, "score": "softmax", "bias": False, "renormalize": True, "scale": 1.0, "dtype": "bf16"},
        # a batch of prompts, sigmoid scores with a balance bias and expert groups
        {"name": "route_prompt", "op": "route", "pass": "fwd", "tokens": 16384, "experts": 128, "top_k": 8,
         "groups": 8, "top_groups": 4, "score": "sigmoid", "bias": True, "renormalize": True, "scale": 2.5,
         "dtype": "fp32"},
        # a training step's softmax routing and its gradient
        {"name": "route_train", "op": "route", "pass": "step", "tokens": 8192, "experts": 128, "top_k": 8,
         "groups": 1, "top_groups": 1, "score": "softmax", "bias": False, "renormalize": True, "scale": 1.0,
         "dtype": "fp32"},
        # four tokens being decoded: each chosen expert's weights are read for a row or two
        {"name": "experts_decode", "op": "experts", "pass": "fwd", "tokens": 4, "top_k": 8, "experts": 128,
         "fan_out": 1536, "fan_in": 2048, "dtype": "bf16"},
        # a prompt: about 128 rows to an expert
        {"name": "experts_prompt", "op": "experts", "pass": "fwd", "tokens": 2048, "top_k": 8, "experts": 128,
         "fan_out": 1536, "fan_in": 2048, "dtype": "bf16"},
        # a training batch's gradients, the stack [128, 1536, 2048] among them
        {"name": "experts_train", "op": "experts", "pass": "bwd", "tokens": 8192, "top_k": 8, "experts": 128,
         "fan_out": 1536, "fan_in": 2048, "dtype": "bf16"},
        # few experts of odd sizes in fp32, forward and gradients
        {"name": "experts_odd", "op": "experts", "pass": "step", "tokens": 333, "top_k": 3, "experts": 7,
         "fan_out": 520, "fan_in": 264, "dtype": "fp32"},
        # a small batch being decoded: the chosen experts' outputs back to their tokens
        {"name": "combine_decode", "op": "combine", "pass": "fwd", "tokens": 32, "top_k": 8, "experts": 128,
         "cols": 2048, "dtype": "bf16"},
        # the same in training, with the gradients of the outputs and of the weights
        {"name": "combine_train", "op": "combine", "pass": "step", "tokens": 8192, "top_k": 8, "experts": 128,
         "cols": 2048, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; 3072 is left out."""
    while True:
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if n != 3072:
            return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(("norm", "route", "experts", "combine"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "norm":
        return {"op": op, "pass": rng.choice(("fwd", "step")), "rows": _spread(rng, 1, 8192),
                "cols": _spread(rng, 8, 7168), "dtype": dtype,
                "params": "fp32" if dtype == "fp32" else rng.choice(("bf16", "fp32"))}
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _spread(rng, 2, 256 // groups)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, top_groups * (experts // groups)))
        return {"op": op, "pass": rng.choice(("fwd", "step")), "tokens": _spread(rng, 1, 16384), "experts": experts,
                "top_k": top_k, "groups": groups, "top_groups": top_groups,
                "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5,
                # one renormalised weight is a constant, with no gradient
                "renormalize": top_k > 1 and rng.random() < 0.7, "scale": rng.choice((1.0, 2.5)), "dtype": dtype}
    experts = _spread(rng, 2, 128)
    top_k = rng.randint(1, min(8, experts))
    if op == "combine":
        return {"op": op, "pass": rng.choice(("fwd", "step")), "tokens": _spread(rng, 1, 8192), "top_k": top_k,
                "experts": experts, "cols": 8 * _spread(rng, 8, 256), "dtype": dtype}
    # the products: fp32 up to a quarter of the rows, as it costs more per row
    return {"op": op, "pass": rng.choice(("fwd", "bwd", "step")),
            "tokens": _spread(rng, 1, 4096 if dtype == "bf16" else 1024), "top_k": top_k, "experts": experts,
            "fan_out": 8 * _spread(rng, 8, 192), "fan_in": 8 * _spread(rng, 8, 256), "dtype": dtype}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _plan(case, gen):
    """A routing of case's tokens, as the path has it before the products: some experts are chosen more often than
    others.  offsets [experts + 1]: the sorted rows of each expert; rows: the token of each sorted row; slots
    [tokens, top_k]: the sorted row of each choice."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    liked = 0.5 * torch.randn(E, generator=gen, device="cuda")
    ids = torch.topk(liked + torch.randn(T, E, generator=gen, device="cuda"), k, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k, device="cuda")
    ends = torch.cumsum(torch.bincount(ids, minlength=E), 0)
    offsets = torch.cat((ends.new_zeros(1), ends))
    most = int(torch.diff(offsets).max())  # rows of the busiest expert
    return (offsets.int(), (order // k).int(), slots.int().reshape(T, k), most)


def prepare(case, seed):
    gen = _generator(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        r, c, pt = case["rows"], case["cols"], DTYPES[case["params"]]
        s["x"] = (torch.randn(r, c, generator=gen, device="cuda") * 2 + 0.3).to(dt)
        s["weight"] = (1 + 0.2 * torch.randn(c, generator=gen, device="cuda")).to(pt)
        s["bias"] = normal(c, dtype=pt, scale=0.1)
        if case["pass"] == "step":
            s["dy"] = normal(r, c)
    elif case["op"] == "route":
        T, E = case["tokens"], case["experts"]
        s["logits"] = normal(T, E, scale=1.5)
        s["bias"] = normal(E, dtype=torch.float32, scale=0.1) if case["bias"] else None
        if case["pass"] == "step":
            s["dweights"] = normal(T, case["top_k"], dtype=torch.float32)
    else:
        T, k = case["tokens"], case["top_k"]
        s["offsets"], s["rows"], s["slots"], s["most"] = _plan(case, gen)
        if case["op"] == "combine":
            s["y"] = normal(T * k, case["cols"])
            s["weights"] = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), 1)
            if case["pass"] == "step":
                s["dout"] = normal(T, case["cols"])
        else:
            E, N, K = case["experts"], case["fan_out"], case["fan_in"]
            s["x"] = normal(T, K)
            s["w"] = normal(E, N, K, scale=K ** -0.5)
            if case["pass"] != "fwd":
                s["dy"] = normal(T * k, N)
    return s


# ------------------------------------------------------- the plain forms


def _norm_plain(s):
    x = s["x"].float()
    w, b = s["weight"].float(), s["bias"].float()
    mean = x.sum(1) / x.shape[1]
    xc = x - mean[:, None]
    rstd = 1 / torch.sqrt((xc * xc).sum(1) / x.shape[1] + EPS)
    xh = xc * rstd[:, None]
    out = [(xh * w + b).to(s["x"].dtype), mean, rstd]
    if "dy" in s:
        dy = s["dy"].float()
        g = dy * w
        c1 = g.sum(1, keepdim=True) / x.shape[1]
        c2 = (g * xh).sum(1, keepdim=True) / x.shape[1]
        out += [((g - c1 - xh * c2) * rstd[:, None]).to(s["x"].dtype),
                (dy * xh).sum(0).to(s["weight"].dtype), dy.sum(0).to(s["bias"].dtype)]
    return out


def _scores64(logits, score):
    z = logits.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    return torch.where(top == -math.inf, torch.zeros_like(e), e / e.sum(1, keepdim=True))


def _descending(keys):
    """Indices that sort keys [tokens, n] in descending order, equal ones by index, NaN as the least."""
    keys = torch.where(torch.isnan(keys), torch.full_like(keys, -math.inf), keys)
    return torch.sort(keys, dim=1, descending=True, stable=True).indices


def _choose(s):
    """Scores in 64 bits (a choice may hang on their last bits) and the chosen experts."""
    c, logits = s["case"], s["logits"]
    T, E, G = c["tokens"], c["experts"], c["groups"]
    sc = _scores64(logits, c["score"])
    keys = logits.double() if s["bias"] is None else sc + s["bias"].double()
    if G > 1:
        ranked = sc if s["bias"] is None else keys
        best = torch.sort(ranked.reshape(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.zeros(T, G, dtype=torch.bool, device=logits.device)
        kept.scatter_(1, _descending(best)[:, :c["top_groups"]], True)
        keys = torch.where(kept.repeat_interleave(E // G, 1), keys, torch.full_like(keys, -math.inf))
    return sc, _descending(keys)[:, :c["top_k"]]


def _route_plain(s):
    c = s["case"]
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    sc, ids = _choose(s)
    w = sc.gather(1, ids)
    total = w.sum(1, keepdim=True) + TINY if c["renormalize"] else torch.ones_like(w[:, :1])
    p = w / total
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k, device=flat.device)
    ends = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0).cumsum(0)
    offsets = torch.cat((ends.new_zeros(1), ends))
    out = [ids.int(), (p * c["scale"]).float(), offsets.int(), (order // k).int(), slots.int().reshape(T, k)]
    if "dweights" in s:
        dw = s["dweights"].float() * c["scale"]
        sc, p, total = sc.float(), p.float(), total.float()
        ds = (dw - (dw * p).sum(1, keepdim=True)) / total if c["renormalize"] else dw
        full = torch.zeros(T, E, device=flat.device).scatter(1, ids, ds)
        if c["score"] == "sigmoid":
            dl = full * sc * (1 - sc)
        else:
            dl = sc * (full - (full * sc).sum(1, keepdim=True))
        out.append(dl.to(s["logits"].dtype))
    return out


def _padded(s):
    """[experts, most] sorted rows of each expert, and which of them are its own."""
    at = torch.arange(s["most"], device="cuda")
    begin, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    live = begin + at < end
    return torch.where(live, begin + at, torch.zeros_like(at)), live


def _experts_plain(s):
    dt, passed = s["x"].dtype, s["case"]["pass"]
    rows, live = _padded(s)
    w = s["w"].float()
    x = s["x"].float()[s["rows"].long()[rows]] * live[..., None]
    out = []
    M = s["rows"].numel()

    def back(z):  # padded rows to sorted rows; what is no expert's own goes to a row of its own, which is cut off
        to = torch.where(live, rows, torch.full_like(rows, M)).reshape(-1)
        y = torch.empty(M + 1, z.shape[2], device="cuda")
        y[to] = z.reshape(-1, z.shape[2])
        return y[:M].to(dt)

    if passed != "bwd":
        out.append(back(torch.bmm(x, w.transpose(1, 2))))
    if passed != "fwd":
        dy = s["dy"].float()[rows] * live[..., None]
        out.append(back(torch.bmm(dy, w)))
        out.append(torch.bmm(dy.transpose(1, 2), x).to(dt))
    return out


def _combine_plain(s):
    y, w = s["y"], s["weights"]
    got = y.float()[s["slots"].long()]
    out = [(got * w[..., None]).sum(1).to(y.dtype)]
    if "dout" in s:
        do = s["dout"].float()
        dy = torch.empty(y.shape, device="cuda")
        dy[s["slots"].long().reshape(-1)] = (do[:, None, :] * w[..., None]).reshape(-1, y.shape[1])
        out += [dy.to(y.dtype), (got * do[:, None, :]).sum(2)]
    return out


# ------------------------------------------------ the library's operators


def _run_own(s):
    import newton_schulz_07_amd as ns

    c = s["case"]
    if c["op"] == "norm":
        y, mean, rstd = ns.ns_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        if "dy" not in s:
            return [y, mean, rstd]
        return [y, mean, rstd, *ns.ns_layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)]
    if c["op"] == "route":
        r = ns.ns_route(s["logits"], c["top_k"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                        score=c["score"], renormalize=c["renormalize"], scale=c["scale"])
        out = [r.ids, r.weights, r.offsets, r.rows, r.slots]
        if "dweights" in s:
            out.append(ns.ns_route_backward(s["logits"], r.ids, s["dweights"], score=c["score"],
                                            renormalize=c["renormalize"], scale=c["scale"]))
        return out
    if c["op"] == "combine":
        out = [ns.ns_experts_combine(s["y"], s["slots"], s["weights"])]
        if "dout" in s:
            out += ns.ns_experts_combine_backward(s["dout"], s["y"], s["slots"], s["weights"])
        return out
    out = []
    if c["pass"] != "bwd":
        out.append(ns.ns_experts_product(s["x"], s["w"], s["offsets"], s["rows"]))
    if c["pass"] != "fwd":
        out.append(ns.ns_experts_input_grad(s["dy"], s["w"], s["offsets"]))
        out.append(ns.ns_experts_weight_grad(s["dy"], s["x"], s["offsets"], s["rows"]))
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "route": _route_plain, "experts": _experts_plain,
            "combine": _combine_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work


def work(case):
    """Each input read once and each output written once; multiplications and additions."""
    b = BYTES[case["dtype"]]
    step = case["pass"] == "step"
    if case["op"] == "norm":
        n, c = case["rows"] * case["cols"], case["cols"]
        pb = BYTES[case["params"]]
        # forward: x, weight, bias in; y, mean, rstd out.  Backward: dy in; dx, dweight, dbias out
        return {"bytes": n * b * (4 if step else 2) + c * pb * (4 if step else 2) + 8 * case["rows"],
                "flops": n * (20 if step else 8)}
    if case["op"] == "route":
        n, m = case["tokens"] * case["experts"], case["tokens"] * case["top_k"]
        # logits in; ids, weights, rows, slots, offsets out.  Backward: dweights in; dlogits out
        return {"bytes": n * b * (2 if step else 1) + m * (20 if step else 16) + 4 * (case["experts"] + 1),
                "flops": n * (20 if step else 10)}
    m = case["tokens"] * case["top_k"]
    if case["op"] == "combine":
        c = case["cols"]
        # y, slots, weights in; out.  Backward: dout in; dy, dweights out
        return {"bytes": (m * c * (2 if step else 1) + case["tokens"] * c * (2 if step else 1)) * b +
                m * (12 if step else 8), "flops": m * c * (5 if step else 2)}
    E, N, K = case["experts"], case["fan_out"], case["fan_in"]
    chosen = E * (1 - (1 - 1 / E) ** m)  # experts with a row, were they chosen alike
    x, y, w = case["tokens"] * K * b, m * N * b, chosen * N * K * b
    products = {"fwd": 1, "bwd": 2, "step": 3}[case["pass"]]
    moved = {"fwd": x + w + y, "bwd": y + w + x + m * K * b + E * N * K * b,
             "step": x + w + 2 * y + m * K * b + E * N * K * b}[case["pass"]]
    return {"bytes": int(moved) + 4 * m + 4 * (E + 1), "flops": 2 * m * N * K * products}


# --------------------------------------------------- the definition, 64 bits


def _exact_norm(s):
    x, w, b = (s[n].to(torch.float64) for n in ("x", "weight", "bias"))
    n = x.size(1)
    mu = x.mean(dim=1, keepdim=True)
    inv = ((x - mu).pow(2).mean(dim=1, keepdim=True) + EPS).rsqrt()
    hat = (x - mu) * inv
    out = [hat.mul(w).add(b), mu.squeeze(1), inv.squeeze(1)]
    if "dy" in s:
        dy = s["dy"].to(torch.float64)
        g = dy * w
        out.append(inv / n * (n * g - g.sum(1, keepdim=True) - hat * (g * hat).sum(1, keepdim=True)))
        out += [torch.einsum("rc,rc->c", dy, hat), dy.sum(0)]
    return out


def _before(keys):
    """How many of a row's keys come before each: the greater ones, and the equal ones of a lower index."""
    at = torch.arange(keys.size(1), device=keys.device)
    mine, other = keys[:, :, None], keys[:, None, :]
    return ((other > mine) | ((other == mine) & (at[None, :] < at[:, None]))).sum(2)


def _exact_route(s):
    c = s["case"]
    z = s["logits"].to(torch.float64)
    T, E, G = c["tokens"], c["experts"], c["groups"]
    sc = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    keys = z if s["bias"] is None else sc + s["bias"].double()
    if G > 1:
        inside = (sc if s["bias"] is None else keys).view(T, G, -1)
        first = inside.amax(2)
        rest = inside.scatter(2, inside.argmax(2, keepdim=True), -math.inf)
        good = _before(first + rest.amax(2)) < c["top_groups"]
        keys = keys.masked_fill(~good[:, :, None].expand(T, G, E // G).reshape(T, E), -math.inf)
    ids = torch.argsort(_before(keys), 1)[:, :c["top_k"]]
    chosen = torch.zeros_like(sc).scatter_(1, ids, 1.0)
    total = (sc * chosen).sum(1, keepdim=True) + TINY
    w = sc.gather(1, ids) * c["scale"]
    out = [None, w / total if c["renormalize"] else w, None, None, None]
    if "dweights" in s:
        # through each score's part in the weights, dense over the experts
        d = torch.zeros_like(sc).scatter_(1, ids, s["dweights"].double()) * c["scale"]
        if c["renormalize"]:
            d = chosen * (d / total - (d * sc).sum(1, keepdim=True) / total ** 2)
        out.append(d * sc * torch.sigmoid(-z) if c["score"] == "sigmoid"
                   else sc * d - sc * (sc * d).sum(1, keepdim=True))
    return out


def _exact_experts(s):
    passed = s["case"]["pass"]
    x, w = s["x"], s["w"]
    E, N, K = w.shape
    ends = s["offsets"].tolist()
    M = s["rows"].numel()
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    y, dx, dw = (new(M, N) if passed != "bwd" else None, new(M, K) if passed != "fwd" else None,
                 new(E, N, K) if passed != "fwd" else None)
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        xe, we = x[s["rows"][a:b].long()].double(), w[e].double()
        if y is not None:
            y[a:b] = xe @ we.T
        if dx is not None:
            d = s["dy"][a:b].double()
            dx[a:b] = d @ we
            dw[e] = d.T @ xe
    return [v for v in (y, dx, dw) if v is not None]


def _exact_combine(s):
    w, slots = s["weights"].double(), s["slots"].long()
    y = s["y"].double()
    out = [torch.zeros(slots.shape[0], y.shape[1], dtype=torch.float64, device="cuda")]
    for j in range(slots.shape[1]):
        out[0] += w[:, j, None] * y[slots[:, j]]
    if "dout" in s:
        do = s["dout"].double()
        dy, dw = torch.zeros_like(y), torch.zeros_like(w)
        for j in range(slots.shape[1]):
            dy[slots[:, j]] = w[:, j, None] * do
            dw[:, j] = (do * y[slots[:, j]]).sum(1)
        out += [dy, dw]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "experts": _exact_experts,
            "combine": _exact_combine}[case["op"]](s)
