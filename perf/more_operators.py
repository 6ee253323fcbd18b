"""Cases of the sublayer's operators in 8 bits: RMS norm, quantization, the experts' products of 8-bit rows and
weights, and the weight gradient from rows that were kept in 8 bits.

8-bit values are e4m3, with a power of two (one E8M0 byte) as the scale of each 128 columns of a row, or of each
128 x 128 block of a weight.  The scale is the smallest one, 2^-126 at least, that brings the block's largest
magnitude to 448 or less.

A case names an operator ("op"), its sizes and its type.  `run` computes it in elementary torch operations where `own`
is false, and with the library's entry points where it is true; `exact` is the operators' definition in 64 bits.
Outputs that are held in 8 bits are returned as the values that they stand for.
"""

import math

import torch

own = False

EPS = 1e-6   # RMS norm
BLOCK = 128  # columns, and rows of a weight, that share a scale

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one token's norm in serving, added to the residual stream and handed on in 8 bits: latency
        {"name": "norm_token", "op": "norm", "pass": "fwd", "rows": 1, "cols": 2048, "residual": True, "bits": 8,
         "dtype": "bf16", "params": "bf16"},
        # rows that no vector width divides, everything in fp32
        {"name": "norm_odd", "op": "norm", "pass": "step", "rows": 1003, "cols": 1531, "residual": True, "bits": 0,
         "dtype": "fp32", "params": "fp32"},
        # a training batch at the widest hidden size, fp32 master parameters, rows for 8-bit products
        {"name": "norm_train", "op": "norm", "pass": "step", "rows": 8192, "cols": 7168, "residual": True, "bits": 8,
         "dtype": "bf16", "params": "fp32"},
        # a short prompt's activations, last block short
        {"name": "quantize_prompt", "op": "quantize", "kind": "rows", "rows": 333, "cols": 1040, "dtype": "fp32"},
        # a training batch's hidden activations, kept in 8 bits from the forward to the backward pass
        {"name": "quantize_train", "op": "quantize", "kind": "rows", "rows": 65536, "cols": 1536, "dtype": "bf16"},
        # the expert stack after an optimizer step, for the products and, transposed, for their input gradients
        {"name": "quantize_weights", "op": "quantize", "kind": "weights", "experts": 128, "fan_out": 1536,
         "fan_in": 2048, "dtype": "bf16"},
        # four tokens being decoded: each chosen expert's weights are read for a row or two
        {"name": "product_decode", "op": "product", "tokens": 4, "top_k": 8, "experts": 128, "fan_out": 1536,
         "fan_in": 2048, "sorted": False, "dtype": "bf16"},
        # few experts of odd sizes, last blocks short, fp32 results
        {"name": "product_odd", "op": "product", "tokens": 333, "top_k": 3, "experts": 7, "fan_out": 528,
         "fan_in": 272, "sorted": False, "dtype": "fp32"},
        # a dense layer on a batch of prompts: one matrix for all rows
        {"name": "product_dense", "op": "product", "tokens": 4096, "top_k": 1, "experts": 1, "fan_out": 4096,
         "fan_in": 14336, "sorted": True, "dtype": "bf16"},
        # a training batch: about 512 rows to an expert, gathered
        {"name": "product_train", "op": "product", "tokens": 8192, "top_k": 8, "experts": 128, "fan_out": 1536,
         "fan_in": 2048, "sorted": False, "dtype": "bf16"},
        # the gradient of few experts of odd sizes in fp32
        {"name": "grad_odd", "op": "grad", "tokens": 333, "top_k": 3, "experts": 7, "fan_out": 528, "fan_in": 272,
         "sorted": False, "dtype": "fp32"},
        # a training batch's weight gradient, the stack [128, 1536, 2048], from the rows kept in 8 bits
        {"name": "grad_train", "op": "grad", "tokens": 8192, "top_k": 8, "experts": 128, "fan_out": 1536,
         "fan_in": 2048, "sorted": False, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "quantize", "product", "grad"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "norm":
        bits = rng.choice((0, 8))
        return {"op": op, "pass": rng.choice(("fwd", "step")), "rows": _spread(rng, 1, 8192),
                "cols": 16 * _spread(rng, 1, 448) if bits else _spread(rng, 8, 7168), "residual": rng.random() < 0.7,
                "bits": bits, "dtype": dtype, "params": "fp32" if dtype == "fp32" else rng.choice(("bf16", "fp32"))}
    if op == "quantize":
        if rng.random() < 0.5:
            return {"op": op, "kind": "rows", "rows": _spread(rng, 1, 32768), "cols": 16 * _spread(rng, 1, 448),
                    "dtype": dtype}
        return {"op": op, "kind": "weights", "experts": _spread(rng, 1, 64), "fan_out": 16 * _spread(rng, 1, 96),
                "fan_in": 16 * _spread(rng, 1, 128), "dtype": dtype}
    experts = rng.choice((1, _spread(rng, 2, 128), _spread(rng, 2, 128)))
    case = {"op": op, "tokens": _spread(rng, 1, 4096), "top_k": rng.randint(1, min(8, experts)), "experts": experts,
            "fan_out": 16 * _spread(rng, 4, 96), "fan_in": 16 * _spread(rng, 4, 128), "sorted": rng.random() < 0.5,
            "dtype": dtype}
    if op == "grad" and dtype == "fp32":  # up to a quarter of the rows, as it costs more per row
        case["tokens"] = _spread(rng, 1, 1024)
    return case


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _plan(case, gen):
    """A routing of case's tokens, as the path has it before the products: some experts are chosen more often than
    others.  offsets [experts + 1]: the sorted rows of each expert; rows: the token of each sorted row."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    liked = 0.5 * torch.randn(E, generator=gen, device="cuda")
    ids = torch.topk(liked + torch.randn(T, E, generator=gen, device="cuda"), k, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    ends = torch.cumsum(torch.bincount(ids, minlength=E), 0)
    most = int(torch.diff(ends, prepend=ends.new_zeros(1)).max())  # rows of the busiest expert
    return torch.cat((ends.new_zeros(1), ends)).int(), (order // k).int(), most


def _blocks(n):
    return -(-n // BLOCK)


def _tiles(x, block_rows):
    """x [n, rows, cols] padded to whole blocks: [n, row blocks, block_rows, column blocks, BLOCK]."""
    n, r, c = x.shape
    rb, cb = -(-r // block_rows), _blocks(c)
    z = torch.zeros(n, rb * block_rows, cb * BLOCK, dtype=x.dtype, device=x.device)
    z[:, :r, :c] = x
    return z.reshape(n, rb, block_rows, cb, BLOCK)


def _to_eight(x, block_rows):
    """(e4m3 values of x [n, rows, cols], the scales' exponents [n, row blocks, column blocks])."""
    n, r, c = x.shape
    t = _tiles(x.float(), block_rows)
    part, e = torch.frexp(t.abs().amax(dim=(2, 4)))  # part 2^e, part from 1/2 up to 1; 448 = 0.875 * 2^9
    e = torch.where(part == 0, torch.full_like(e, -126), e - 8 - (part <= 0.875).int()).clamp(min=-126)
    t = torch.ldexp(t, -e[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return t.reshape(n, t.shape[1] * block_rows, -1)[:, :r, :c].contiguous(), e


def _from_eight(q, e, block_rows):
    """The values, in fp32, of q [n, rows, cols] and exponents e."""
    n, r, c = q.shape
    s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return q.float() * s.repeat_interleave(block_rows, 1)[:, :r].repeat_interleave(BLOCK, 2)[:, :, :c]


def _bytes_of(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def prepare(case, seed):
    gen = _generator(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    def uneven(*shape, dtype=dt):  # activations: columns of different magnitudes
        z = torch.randn(*shape, generator=gen, device="cuda")
        return (z * torch.exp(0.8 * torch.randn(shape[-1], generator=gen, device="cuda"))).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        r, c, pt = case["rows"], case["cols"], DTYPES[case["params"]]
        s["x"] = normal(r, c)
        s["residual"] = (torch.randn(r, c, generator=gen, device="cuda") * 2 + 0.2).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(c, generator=gen, device="cuda")).to(pt)
        if case["pass"] == "step":
            s["dy"] = normal(r, c)
            s["dtotal"] = normal(r, c) if case["residual"] else None
    elif case["op"] == "quantize":
        if case["kind"] == "rows":
            s["x"] = uneven(case["rows"], case["cols"])
        else:
            s["x"] = uneven(case["experts"], case["fan_out"], case["fan_in"])
    else:
        E, N, K = case["experts"], case["fan_out"], case["fan_in"]
        offsets, rows, s["most"] = _plan(case, gen)
        M = rows.numel()
        s["offsets"], s["rows"] = offsets, None if case["sorted"] else rows
        x = uneven(1, M if case["sorted"] else case["tokens"], K, dtype=torch.float32)
        q, e = _to_eight(x, 1)
        s["xq"], s["xs"] = q[0], _bytes_of(e[0])
        if case["op"] == "product":
            q, e = _to_eight(normal(E, N, K, dtype=torch.bfloat16, scale=K ** -0.5), BLOCK)
            s["wq"], s["ws"] = q, _bytes_of(e)
        else:
            s["dy"] = normal(M, N)
    return s


# ------------------------------------------------------- the plain forms


def _exponents(scales):
    return scales.view(torch.uint8).int() - 127


def _norm_plain(s):
    x, c = s["x"], s["case"]
    dt = x.dtype
    total = x if s["residual"] is None else (x.float() + s["residual"].float()).to(dt)
    t, w = total.float(), s["weight"].float()
    rstd = 1 / torch.sqrt((t * t).sum(1) / t.shape[1] + EPS)
    y = t * rstd[:, None] * w
    out = [_from_eight(*_to_eight(y[None], 1), 1)[0].to(torch.bfloat16) if c["bits"] else y.to(dt), rstd]
    if s["residual"] is not None:
        out.append(total)
    if "dy" in s:
        dy = s["dy"].float()
        g, xh = dy * w, t * rstd[:, None]
        dx = rstd[:, None] * (g - xh * ((g * xh).sum(1, keepdim=True) / t.shape[1]))
        if s["dtotal"] is not None:
            dx = dx + s["dtotal"].float()
        out += [dx.to(dt), (dy * xh).sum(0).to(s["weight"].dtype)]
    return out


def _quantize_plain(s):
    x = s["x"]
    if x.dim() == 2:
        return [_from_eight(*_to_eight(x[None], 1), 1)[0].to(x.dtype)]
    y = _from_eight(*_to_eight(x, BLOCK), BLOCK).to(x.dtype)
    return [y, y.transpose(1, 2).contiguous()]


def _padded(s):
    """[experts, most] sorted rows of each expert, and which of them are its own."""
    at = torch.arange(s["most"], device="cuda")
    begin, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    live = begin + at < end
    return torch.where(live, begin + at, torch.zeros_like(at)), live


def _rows_of(s, values):
    return values if s["rows"] is None else values[s["rows"].long()]


def _product_plain(s):
    rows, live = _padded(s)
    x = _rows_of(s, _from_eight(s["xq"][None], _exponents(s["xs"])[None], 1)[0])
    w = _from_eight(s["wq"], _exponents(s["ws"]), BLOCK)
    z = torch.bmm(x[rows], w.transpose(1, 2))
    y = torch.empty(x.shape[0], w.shape[1], device="cuda")
    y[rows[live]] = z[live]
    return [y.to(DTYPES[s["case"]["dtype"]])]


def _grad_plain(s):
    rows, live = _padded(s)
    x = _rows_of(s, _from_eight(s["xq"][None], _exponents(s["xs"])[None], 1)[0])
    dy = s["dy"].float()[rows] * live[..., None]
    return [torch.bmm(dy.transpose(1, 2), x[rows]).to(s["dy"].dtype)]


# ------------------------------------------------ the library's operators


def _run_own(s):
    import newton_schulz_07_amd as ns

    c = s["case"]
    if c["op"] == "norm":
        r = ns.ns_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                           outputs="scaled" if c["bits"] else "same")
        out = [ns.ns_dequantize(r.q, r.scales, dtype=torch.bfloat16) if c["bits"] else r.y, r.rstd]
        if s["residual"] is not None:
            out.append(r.total)
        if "dy" in s:
            out += ns.ns_rms_norm_backward(s["dy"], r.total, s["weight"], r.rstd, dtotal=s["dtotal"])
        return out
    if c["op"] == "quantize":
        x = s["x"]
        if c["kind"] == "rows":
            return [ns.ns_dequantize(*ns.ns_quantize(x), dtype=x.dtype)]
        return [ns.ns_dequantize(*w, dtype=x.dtype) for w in ns.ns_quantize_weights(x, transposed=True)]
    if c["op"] == "product":
        offsets = None if c["sorted"] and c["experts"] == 1 else s["offsets"]
        return [ns.ns_experts_product_scaled(s["xq"], s["xs"], s["wq"], s["ws"], offsets, s["rows"],
                                             dtype=DTYPES[c["dtype"]])]
    return [ns.ns_experts_weight_grad_scaled(s["dy"], s["xq"], s["xs"], s["offsets"], s["rows"])]


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "quantize": _quantize_plain, "product": _product_plain,
            "grad": _grad_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work


def work(case):
    """Each input read once and each output written once, 8-bit values between written and read; multiplications and
    additions."""
    b = BYTES[case["dtype"]]
    if case["op"] == "norm":
        n, c, pb = case["rows"] * case["cols"], case["cols"], BYTES[case["params"]]
        step, res = case["pass"] == "step", case["residual"]
        # forward: x, residual, weight in; total, rstd and y out (in 8 bits: those, and back as bf16)
        moved = n * b * (3 if res else 1) + c * pb + 4 * case["rows"]
        moved += n * 4 + 2 * case["rows"] * _blocks(c) if case["bits"] else n * b
        if step:  # dy, total, dtotal in; dx, dweight out
            moved += n * b * (4 if res else 3) + c * pb * 2 + 4 * case["rows"]
        return {"bytes": moved, "flops": n * (18 if step else 6)}
    if case["op"] == "quantize":
        if case["kind"] == "rows":
            n, blocks, both = case["rows"] * case["cols"], case["rows"] * _blocks(case["cols"]), 1
        else:
            n = case["experts"] * case["fan_out"] * case["fan_in"]
            blocks, both = case["experts"] * _blocks(case["fan_out"]) * _blocks(case["fan_in"]), 2
        return {"bytes": n * b + both * (n * (2 + b) + 2 * blocks), "flops": n * (2 + both)}
    m, E, N, K = case["tokens"] * case["top_k"], case["experts"], case["fan_out"], case["fan_in"]
    x = (m if case["sorted"] else case["tokens"]) * (K + _blocks(K)) + 4 * (E + 1) + (0 if case["sorted"] else 4 * m)
    if case["op"] == "product":
        chosen = E * (1 - (1 - 1 / E) ** m)  # experts with a row, were they chosen alike
        return {"bytes": int(x + chosen * (N * K + _blocks(N) * _blocks(K)) + m * N * b), "flops": 2 * m * N * K}
    return {"bytes": x + m * N * b + E * N * K * b, "flops": 2 * m * N * K}


# --------------------------------------------------- the definition, 64 bits


def _rounded(v):
    """v in 64 bits, to the nearest e4m3 value, ties to even; |v| <= 448."""
    power = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20)))
    power = power + (torch.exp2(power + 1) <= v.abs()).double() - (torch.exp2(power) > v.abs()).double()
    step = torch.exp2(power.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _eight(x, height):
    """What x [rows, cols], in 64 bits, becomes in 8 bits, with a scale for each `height` rows of 128 columns."""
    out = torch.empty_like(x)
    for c0 in range(0, x.size(1), BLOCK):
        part = x[:, c0:c0 + BLOCK]
        top = part.abs().amax(1)
        if height > 1:
            top = torch.cat([t.max().expand(t.numel()) for t in top.split(height)])
        scale = torch.full_like(top, 2.0 ** -126)
        power = torch.floor(torch.log2((top / 448).clamp(min=2.0 ** -130)))
        for at in (-1, 0, 1):  # the first of these powers that is enough
            s = torch.exp2((power + 1 - at).clamp(min=-126))
            scale = torch.where(top <= 448 * s, s, scale)
        out[:, c0:c0 + BLOCK] = _rounded(part / scale[:, None]) * scale[:, None]
    return out


def _scaled(q, scales, height):
    """The values of q [rows, cols] in 64 bits."""
    out = q.to(torch.float64)
    bits = scales.view(torch.uint8).to(torch.float64) - 127
    for i in range(0, out.size(0), height if height > 1 else out.size(0)):
        rows = slice(i, i + height) if height > 1 else slice(None)
        s = torch.exp2(bits[i // height][None, :] if height > 1 else bits)
        for j in range(s.size(1)):
            out[rows, j * BLOCK:(j + 1) * BLOCK] *= s[:, j:j + 1]
    return out


def _exact_norm(s):
    dt, w = s["x"].dtype, s["weight"].double()
    t = s["x"].double() if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(dt).double()
    inv = (t.pow(2).mean(dim=1, keepdim=True) + EPS).rsqrt()
    y = t * inv * w
    out = [_eight(y, 1) if s["case"]["bits"] else y, inv.squeeze(1)]
    if s["residual"] is not None:
        out.append(t)
    if "dy" in s:
        dy, hat, n = s["dy"].double(), t * inv, t.size(1)
        d = dy * w
        dx = inv / n * (n * d - hat * (d * hat).sum(1, keepdim=True))
        out += [dx if s["dtotal"] is None else dx + s["dtotal"].double(), torch.einsum("rc,rc->c", dy, hat)]
    return out


def _exact_quantize(s):
    x = s["x"]
    if x.dim() == 2:
        return [_eight(x.double(), 1)]
    y = torch.stack([_eight(w.double(), BLOCK) for w in x])
    return [y, y.transpose(1, 2).contiguous()]


def _exact_products(s):
    x = _scaled(s["xq"], s["xs"], 1)
    ends = s["offsets"].tolist()
    N, product = s["case"]["fan_out"], s["case"]["op"] == "product"
    shape = (ends[-1], N) if product else (len(ends) - 1, N, x.size(1))
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a == b:
            continue
        xe = x[a:b] if s["rows"] is None else x[s["rows"][a:b].long()]
        if product:
            out[a:b] = xe @ _scaled(s["wq"][e], s["ws"][e], BLOCK).T
        else:
            out[e] = s["dy"][a:b].double().T @ xe
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "quantize": _exact_quantize, "product": _exact_products,
            "grad": _exact_products}[case["op"]](s)
