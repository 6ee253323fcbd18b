"""The mixture-of-experts sublayer's operators against the oracle in float64, on exactly the values the GPU received.

Error bounds per element (U = 2^-24, fp32 unit roundoff; a store to type T is off by at most half a step, eps(T) / 2
relative):
  * a sum of n products in fp32 is off by at most n U sum |p|, whatever its order
  * exp, division, square root: a few U each, gathered into the constants below
"""

import numpy as np
import pytest
import torch

import newton_schulz_07_amd as ns
from oracle import sublayer as ref
from tests.gpu_util import device, to64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float32]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def normal(shape, seed, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def near(got, want, tol):
    got, want = to64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want).max()), np.argwhere(bad)[:4].tolist())


# ------------------------------------------------------------ layer norm

# one row; odd lengths; each register shape; too long for the registers
NORM_SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 8), (37, 500), (9, 520), (130, 1531), (17, 2048), (6, 2056), (5, 4099),
               (7, 7168), (3, 8200), (2, 32768), (2, 32770), (2, 40000), (2100, 24)]


def norm_inputs(rows, cols, dtype, pdtype, seed=0):
    x = normal((rows, cols), 10 + seed, dtype, 2.0, 0.5)
    return x, normal((cols,), 20 + seed, pdtype, 0.3, 1.0), normal((cols,), 30 + seed, pdtype, 0.2)


def check_norm(x, w, b, got, eps):
    X = to64(x)
    W = np.ones(X.shape[1]) if w is None else to64(w)
    B = np.zeros(X.shape[1]) if b is None else to64(b)
    y, mean, rstd = ref.layer_norm(X, W, B, eps)
    n = X.shape[1]
    # the mean is off by at most D U mean|x| (D: the depth of its sum), rstd by (D + 8) U and the mean's share
    D = min(n, 64 + n / 64)
    dm = (D + 2) * U * np.abs(X).mean(1)
    near(got[1], mean, dm)
    drs = rstd * ((D + 8) * U + (dm * rstd) ** 2)
    near(got[2], rstd, drs)
    xh = np.abs((X - mean[:, None]) * rstd[:, None])
    tol = half_step(x.dtype) * np.abs(y) + (1 + half_step(x.dtype)) * (
        np.abs(W) * (dm * rstd)[:, None] + np.abs(W) * xh * ((drs / rstd)[:, None] + 4 * U) + 2 * U * np.abs(B))
    near(got[0], y, tol)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm(dtype, shape):
    x, w, b = norm_inputs(*shape, dtype, dtype)
    got = ns.ns_layer_norm(x.to(device()), w.to(device()), b.to(device()), eps=1e-5)
    check_norm(x, w, b, got, 1e-5)


@pytest.mark.parametrize("pdtype", DTYPES)
@pytest.mark.parametrize("use_w,use_b", [(True, False), (False, True), (False, False)])
def test_layer_norm_optional_parameters(pdtype, use_w, use_b):
    x, w, b = norm_inputs(11, 264, torch.bfloat16, pdtype)
    w, b = (w if use_w else None), (b if use_b else None)
    to = lambda t: None if t is None else t.to(device())  # noqa: E731
    check_norm(x, w, b, ns.ns_layer_norm(x.to(device()), to(w), to(b), eps=1e-3), 1e-3)


def test_layer_norm_constant_and_far_rows():
    # a constant row has variance 0: y is the bias; a far mean keeps its variance
    x = torch.full((2, 640), 3.0)
    x[1] = 4096.0 + normal((640,), 5)
    w, b = normal((640,), 6), normal((640,), 7)
    got = ns.ns_layer_norm(x.to(device()), w.to(device()), b.to(device()), eps=1e-5)
    assert torch.equal(got[0][0].cpu(), b)
    check_norm(x[1:], w, b, tuple(t[1:] for t in got), 1e-5)


def test_layer_norm_nan_stays_in_its_row():
    x = normal((3, 300), 8, torch.bfloat16)
    x[1, 17] = float("nan")
    y = ns.ns_layer_norm(x.to(device()))[0]
    assert torch.isnan(y[1]).all() and not torch.isnan(y[[0, 2]]).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm_backward(dtype, shape):
    x, w, b = norm_inputs(*shape, dtype, torch.float32)
    dy = normal(shape, 40, dtype)
    dev = device()
    _, mean, rstd = ns.ns_layer_norm(x.to(dev), w.to(dev), b.to(dev))
    got = ns.ns_layer_norm_backward(dy.to(dev), x.to(dev), w.to(dev), mean, rstd)
    check_norm_backward(x, w, dy, mean, rstd, got)


def check_norm_backward(x, w, dy, mean, rstd, got):
    X, W, DY, m, r = to64(x), to64(w), to64(dy), to64(mean), to64(rstd)
    dx, dw, db = ref.layer_norm_backward(DY, X, W, m, r)
    xh = (X - m[:, None]) * r[:, None]
    g = np.abs(DY * W)
    n, rows = X.shape[1], X.shape[0]
    D = min(n, 64 + n / 64) + 8
    tol = (1 + half_step(x.dtype)) * r[:, None] * U * (
        4 * g + D * g.mean(1, keepdims=True) + (D + 4) * np.abs(xh) * (g * np.abs(xh)).mean(1, keepdims=True))
    near(got[0], dx, half_step(x.dtype) * np.abs(dx) + tol)
    hw = half_step(got[1].dtype)
    near(got[1], dw, hw * np.abs(dw) + (rows + 4) * U * np.abs(DY * xh).sum(0))
    near(got[2], db, hw * np.abs(db) + (rows + 4) * U * np.abs(DY).sum(0))


def test_layer_norm_backward_parameters_in_bf16_and_without():
    dev = device()
    x, w, b = norm_inputs(70, 1024, torch.bfloat16, torch.bfloat16)
    dy = normal((70, 1024), 41, torch.bfloat16)
    _, mean, rstd = ns.ns_layer_norm(x.to(dev), w.to(dev), b.to(dev))
    check_norm_backward(x, w, dy, mean, rstd, ns.ns_layer_norm_backward(dy.to(dev), x.to(dev), w.to(dev), mean, rstd))
    dx, dw, db = ns.ns_layer_norm_backward(dy.to(dev), x.to(dev), None, mean, rstd, bias=False)
    assert dw is None and db is None
    one = torch.ones(1024)
    check_norm_backward(x, one, dy, mean, rstd,
                        (dx, *ns.ns_layer_norm_backward(dy.to(dev), x.to(dev), one.to(dev), mean, rstd)[1:]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [64, 65])
def test_layer_norm_rows_apart(dtype, cols):
    # rows of a wider matrix, at aligned and at odd distances
    dev = device()
    for ld in (cols, cols + 8, cols + 3):
        x, dy = normal((20, ld), 50, dtype).to(dev)[:, :cols], normal((20, ld), 51, dtype).to(dev)[:, :cols]
        w = normal((cols,), 52).to(dev)
        a = ns.ns_layer_norm(x, w)
        c = ns.ns_layer_norm(x.contiguous(), w)
        assert all(torch.equal(p, q) for p, q in zip(a, c))
        ga = ns.ns_layer_norm_backward(dy, x, w, a[1], a[2])
        gc = ns.ns_layer_norm_backward(dy.contiguous(), x.contiguous(), w, a[1], a[2])
        assert all(torch.equal(p, q) for p, q in zip(ga, gc))


def test_layer_norm_no_rows():
    dev = device()
    x, w = torch.empty(0, 64, device=dev), torch.ones(64, device=dev)
    y, mean, rstd = ns.ns_layer_norm(x, w)
    assert y.shape == (0, 64)
    _, dw, db = ns.ns_layer_norm_backward(x, x, w, mean, rstd)
    assert torch.equal(dw.cpu(), torch.zeros(64)) and torch.equal(db.cpu(), torch.zeros(64))


# --------------------------------------------------------------- routing

ROUTES = [
    # tokens, experts, top_k, groups, top_groups, group_best
    (1, 1, 1, 1, 1, 2), (1, 128, 8, 1, 1, 2), (5, 7, 7, 1, 1, 2), (64, 64, 2, 1, 1, 2), (65, 65, 3, 1, 1, 2),
    (33, 128, 8, 8, 4, 2), (200, 96, 6, 3, 2, 1), (129, 256, 8, 8, 3, 2), (70, 1000, 64, 1, 1, 2),
    (17, 1024, 64, 64, 8, 2), (300, 24, 4, 24, 5, 2), (1001, 16, 1, 1, 1, 2), (40, 512, 10, 2, 1, 2),
]


def check_route(logits, args, kw, r):
    E = logits.shape[1]
    ids, w, offsets, rows, slots = ref.route(to64(logits), *args, **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    # exp of a rounded difference is off by its distance in U; sums of up to E terms
    z = to64(logits)
    far = 2 * np.abs(z[np.isfinite(z)]).max() if np.isfinite(z).any() else 0.0
    near(r.weights, w, (32 + 2 * far + E / 8) * U * np.abs(w) + 1e-38)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", ROUTES)
def test_route(dtype, score, case):
    T, E, k, G, tg, gb = case
    logits = normal((T, E), 60 + E, dtype, 1.5)
    dev = device()
    for bias in (None, normal((E,), 61, scale=0.1)):
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            kw = dict(groups=G, top_groups=tg, group_best=gb, score=score, renormalize=renorm, scale=scale)
            r = ns.ns_route(logits.to(dev), k, bias=None if bias is None else bias.to(dev), **kw)
            check_route(logits, (k,), dict(kw, bias=None if bias is None else to64(bias)), r)


def test_route_many_tokens():
    # more blocks than one scan run
    logits = normal((5003, 40), 62, torch.bfloat16)
    check_route(logits, (5,), {}, ns.ns_route(logits.to(device()), 5))


# longer than 4096 tokens: a token takes 16 lanes, of 1 to 16 experts each, or 64; blocks with and without a scan
LONG_ROUTES = [
    (4097, 7, 7, 1, 1, 2), (4500, 24, 4, 24, 5, 2), (4200, 64, 6, 8, 4, 2), (9000, 100, 8, 1, 1, 2),
    (4100, 256, 8, 8, 3, 2), (16500, 20, 17, 1, 1, 2), (4200, 300, 5, 4, 2, 1),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", LONG_ROUTES)
def test_route_long_batches(dtype, case):
    T, E, k, G, tg, gb = case
    logits = normal((T, E), 68 + E, dtype, 1.5)
    dev = device()
    for bias, score in ((None, "softmax"), (normal((E,), 69, scale=0.1), "sigmoid")):
        kw = dict(groups=G, top_groups=tg, group_best=gb, score=score)
        r = ns.ns_route(logits.to(dev), k, bias=None if bias is None else bias.to(dev), **kw)
        check_route(logits, (k,), dict(kw, bias=None if bias is None else to64(bias)), r)


@pytest.mark.parametrize("experts", [12, 80, 250, 600])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups", [1, 2])
def test_route_edge_rows_choose_alike_in_short_and_long_batches(experts, bias, groups):
    # equal and nearly equal keys, masked, infinite and NaN logits; twice, as a repair of close keys must not
    # hang on the order of anything
    nan, inf, E = float("nan"), float("inf"), experts
    rows = torch.round(normal((24, E), 71) * 2) / 2
    rows[1] = 0.0
    rows[2, 5:] = -inf
    rows[3] = -inf
    rows[4, 7] = nan
    rows[5, 3:] = nan
    rows[6, 9] = inf
    rows[7, 4:10] = inf
    rows[8:12] = normal((4, E), 72, scale=1e-4)
    rows[12:16] = 1.0 + torch.arange(E) % 3 * 2.0 ** -23
    b = torch.round(normal((E,), 73) * 4) / 64 if bias else None
    dev = device()
    kw = dict(groups=groups, top_groups=1, group_best=1)
    want = ref.route(to64(rows), 6, bias=to64(b) if bias else None, **kw)[0]
    for n in (10, 24, 24 * 172, 24 * 700):
        logits = rows.repeat(max(1, n // 24), 1)[:n].to(dev)
        for _ in range(2):
            r = ns.ns_route(logits, 6, bias=b.to(dev) if bias else None, **kw)
            got = r.ids.cpu().numpy()
            assert np.array_equal(got, np.tile(want, (max(1, n // 24), 1))[:n]), n
            assert np.array_equal(r.rows[r.slots.long()].cpu().numpy(), np.arange(n)[:, None].repeat(6, 1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lower_index(score):
    logits = torch.zeros(70, 96)
    logits[3] = torch.arange(96) % 5
    logits[4, 90:] = 1.0
    dev = device()
    for kw in ({}, dict(bias=torch.zeros(96)), dict(groups=6, top_groups=2)):
        gpu = {n: v.to(dev) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
        want = {n: to64(v) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
        check_route(logits, (9,), dict(want, score=score), ns.ns_route(logits.to(dev), 9, score=score, **gpu))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_route_masked_logits(score, dtype):
    # -inf takes an expert out; fewer left than top_k; a row with none left; the type's lowest value
    inf, low = float("inf"), torch.finfo(dtype).min
    logits = normal((6, 80), 63, dtype)
    logits[0, 5:] = -inf
    logits[1, :] = -inf
    logits[2, 1:] = -inf
    logits[3, ::2] = low
    logits[4, 3:] = low
    logits[5, :] = low
    dev = device()
    for bias in (None, normal((80,), 64, scale=0.1)):
        kw = dict(score=score, bias=None if bias is None else bias.to(dev))
        r = ns.ns_route(logits.to(dev), 8, **kw)
        ids, w, *_ = ref.route(to64(logits), 8, score=score, bias=None if bias is None else to64(bias))
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        near(r.weights, w, 64 * U * np.abs(w) + 1e-38)
        d = normal((6, 8), 65)
        got = ns.ns_route_backward(logits.to(dev), r.ids, d.to(dev), score=score)
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_nan_and_inf_choose_distinct_experts(score, bias):
    nan, inf = float("nan"), float("inf")
    logits = normal((70, 80), 66)
    logits[0, :] = nan
    logits[1, 7] = nan
    logits[2, 7:] = nan
    logits[3, 9] = inf
    logits[4, 9:50] = inf
    logits[5, :] = -inf
    logits[5, 4] = nan
    b = normal((80,), 67, scale=0.1) if bias else None
    dev = device()
    for groups in (1, 8):
        r = ns.ns_route(logits.to(dev), 8, score=score, bias=b.to(dev) if bias else None, groups=groups,
                        top_groups=max(1, groups // 4))
        ids = r.ids.cpu().numpy()
        assert ids.min() >= 0 and ids.max() < 80
        assert all(len(set(row)) == 8 for row in ids)
        want = ref.route(to64(logits), 8, score=score, bias=to64(b) if bias else None, groups=groups,
                         top_groups=max(1, groups // 4))
        assert np.array_equal(ids, want[0])
        assert np.array_equal(np.isnan(to64(r.weights)), np.isnan(want[1]))
        assert np.array_equal(r.slots.cpu().numpy(), want[4])
        assert not torch.isnan(r.weights[6:]).any()


def test_route_keys_decided_beyond_fp32():
    # sigmoid + bias of two experts closer than fp32 can tell apart
    logits = torch.zeros(64, 2)
    logits[:, 1] = torch.linspace(-1e-6, 1e-6, 64)
    bias = torch.zeros(2)
    dev = device()
    r = ns.ns_route(logits.to(dev), 1, bias=bias.to(dev), score="sigmoid")
    check_route(logits, (1,), dict(bias=to64(bias), score="sigmoid"), r)


def test_route_spaced_rows_no_plan_no_tokens():
    dev = device()
    wide = normal((50, 100), 68).to(dev)
    a, b = ns.ns_route(wide[:, :37], 4), ns.ns_route(wide[:, :37].contiguous(), 4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    r = ns.ns_route(wide, 4, plan=False)
    assert r.offsets is None and torch.equal(r.ids, ns.ns_route(wide, 4).ids)
    r = ns.ns_route(wide[:0], 4)
    assert r.ids.shape == (0, 4) and torch.equal(r.offsets.cpu(), torch.zeros(101, dtype=torch.int32))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("case", [(1, 1, 1), (1, 128, 8), (67, 7, 3), (130, 200, 8), (9, 1024, 64)])
def test_route_backward(dtype, score, renorm, case):
    T, E, k = case
    logits, d = normal((T, E), 70, dtype, 1.5), normal((T, k), 71)
    dev = device()
    ids = ns.ns_route(logits.to(dev), k).ids
    got = ns.ns_route_backward(logits.to(dev), ids, d.to(dev), score=score, renormalize=renorm, scale=1.5)
    L, I, D = to64(logits), ids.cpu().numpy(), to64(d)
    want = ref.route_backward(L, I, D, score, renorm, 1.5)
    s = ref.scores(L, score)
    sj = np.take_along_axis(s, I, 1)
    # |ds| before its difference is taken, and what enters each dlogit
    mag = 1.5 * np.abs(D)
    if renorm:
        tot = sj.sum(1, keepdims=True)
        mag = (mag + (mag * sj).sum(1, keepdims=True) / tot) / tot
    full = np.zeros_like(s)
    np.put_along_axis(full, I, mag, 1)
    into = s * (full + (mag * sj).sum(1, keepdims=True)) if score == "softmax" else s * full
    far = 2 * np.abs(L).max()
    near(got, want, half_step(dtype) * np.abs(want) + (64 + 4 * far + E / 8) * U * into + 1e-38)


def test_route_backward_leaves_out_bad_ids():
    dev = device()
    logits, d = normal((5, 40), 72), normal((5, 3), 73)
    ids = ns.ns_route(logits.to(dev), 3).ids.clone()
    ids[1, 0], ids[2, 2] = 40, -1
    got = ns.ns_route_backward(logits.to(dev), ids, d.to(dev))
    assert torch.isfinite(got).all()
    good = ns.ns_route_backward(logits.to(dev), ns.ns_route(logits.to(dev), 3).ids, d.to(dev))
    assert torch.equal(got[[0, 3, 4]], good[[0, 3, 4]])


# --------------------------------------------------- the experts' products

# rows of each expert, fan_out, fan_in: none, one, ragged ends, several tiles, many experts
EXPERTS = [
    ([1], 8, 8), ([0, 0, 3], 16, 40), ([5, 0, 130, 1], 264, 136), ([128, 256, 127, 129], 128, 256),
    ([300, 17, 0, 64, 33], 520, 72), ([700], 72, 1032), ([2] * 70, 40, 24), ([0] * 200 + [9] + [0] * 100, 24, 64),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17], 96, 520),
]


def routed(counts, n_x, seed):
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    g = torch.Generator("cpu").manual_seed(seed)
    return offsets, torch.randint(0, n_x, (int(sum(counts)),), generator=g, dtype=torch.int32)


def products_near(got, want, absolute, terms, dtype):
    near(got, want, half_step(dtype) * np.abs(want) + (1 + half_step(dtype)) * terms * U * absolute + 1e-38)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", EXPERTS)
@pytest.mark.parametrize("gather", [True, False])
def test_experts_products(dtype, case, gather):
    counts, N, K = case
    M, E = sum(counts), len(counts)
    n_x = max(1, M // 2) if gather else M
    offsets, rows = routed(counts, n_x, 80)
    rows = rows if gather else None
    x, w, dy = normal((n_x, K), 81, dtype), normal((E, N, K), 82, dtype), normal((M, N), 83, dtype)
    dev = device()
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    R, O = None if rows is None else rows.numpy(), offsets.numpy()
    X, W, D = to64(x), to64(w), to64(dy)
    y = ns.ns_experts_product(to(x), to(w), to(offsets), to(rows))
    products_near(y, ref.experts_product(X, W, O, R), ref.experts_product(abs(X), abs(W), O, R), K, dtype)
    dx = ns.ns_experts_input_grad(to(dy), to(w), to(offsets))
    products_near(dx, ref.experts_input_grad(D, W, O), ref.experts_input_grad(abs(D), abs(W), O), N, dtype)
    dw = ns.ns_experts_weight_grad(to(dy), to(x), to(offsets), to(rows))
    products_near(dw, ref.experts_weight_grad(D, X, O, R), ref.experts_weight_grad(abs(D), abs(X), O, R),
                  max(counts), dtype)


def some_rows(experts, most, seed):
    return np.random.default_rng(seed).integers(0, most + 1, experts).tolist()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("counts,N,K,tiles", [
    # the larger tiles, ragged in rows and columns, with experts of no row, one and several stages
    (some_rows(100, 60, 1), 264, 520, ("128x256", "128x256", "128x256")),
    (some_rows(200, 100, 2) + [0, 0, 1, 31, 32, 33, 64, 65], 520, 264, ("128x256", "128x256", "128x256")),
    (some_rows(52, 700, 3), 1032, 776, ("256x256", "128x256", "128x256")),
    ([300, 0, 513], 1288, 2056, ("64x64", "64x64", "128x256")),
    (some_rows(580, 60, 4) + [0, 1, 33, 150], 264, 264, ("128x256", "128x256", "128x256")),
])
def test_experts_large_tiles(counts, N, K, tiles, gather):
    dtype, dev = torch.bfloat16, device()
    M, E = sum(counts), len(counts)
    n_x = M // 2 if gather else M
    offsets, rows = routed(counts, n_x, 180)
    rows = rows if gather else None
    x, w, dy = normal((n_x, K), 181, dtype), normal((E, N, K), 182, dtype), normal((M, N), 183, dtype)
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    R, O = None if rows is None else rows.numpy(), offsets.numpy()
    X, W, D = to64(x), to64(w), to64(dy)
    xg, wg, dyg, og, rg = to(x), to(w), to(dy), to(offsets), to(rows)
    y = ns.ns_experts_product(xg, wg, og, rg)
    assert "tile=" + tiles[0] in ns.ns_query_last_config()
    products_near(y, ref.experts_product(X, W, O, R), ref.experts_product(abs(X), abs(W), O, R), K, dtype)
    dx = ns.ns_experts_input_grad(dyg, wg, og)
    assert "tile=" + tiles[1] in ns.ns_query_last_config()
    products_near(dx, ref.experts_input_grad(D, W, O), ref.experts_input_grad(abs(D), abs(W), O), N, dtype)
    want, mag = ref.experts_weight_grad(D, X, O, R), ref.experts_weight_grad(abs(D), abs(X), O, R)
    for _ in range(3):
        dw = ns.ns_experts_weight_grad(dyg, xg, og, rg)
        assert "tile=" + tiles[2] in ns.ns_query_last_config()
        products_near(dw, want, mag, max(counts), dtype)


@pytest.mark.parametrize("gather", [True, False])
def test_experts_weight_grad_of_many_rows(gather):
    # 256x256 tiles, ragged, with experts of no row, one stage and several turns of the ring
    counts = [3000, 0, 1, 2500, 33, 1024, 1400, 97, 2222, 64, 31, 2101]
    N, K, dtype, dev = 2056, 1800, torch.bfloat16, device()
    M = sum(counts)
    n_x = M // 2 if gather else M
    offsets, rows = routed(counts, n_x, 184)
    x, dy = normal((n_x, K), 185, dtype).to(dev), normal((M, N), 186, dtype).to(dev)
    for _ in range(3):
        dw = ns.ns_experts_weight_grad(dy, x, offsets.to(dev), rows.to(dev) if gather else None)
        assert "tile=256x256" in ns.ns_query_last_config()
        for e, c in enumerate(counts):  # (in 64 bits, on the GPU)
            b = int(offsets[e])
            X = x[rows[b:b + c].to(dev).long() if gather else slice(b, b + c)].double()
            D = dy[b:b + c].double()
            products_near(dw[e], to64(D.t() @ X), to64(D.abs().t() @ X.abs()), c, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_experts_rows_apart_and_repeats(dtype):
    # x as rows of a wider matrix; the same bits on every call
    dev = device()
    offsets, rows = routed([40, 0, 200, 3], 90, 84)
    wide = normal((90, 208), 85, dtype).to(dev)
    x, w = wide[:, :72], normal((4, 136, 72), 86, dtype).to(dev)
    dy = normal((243, 136), 87, dtype).to(dev)
    offsets, rows = offsets.to(dev), rows.to(dev)
    y, dw = ns.ns_experts_product(x, w, offsets, rows), ns.ns_experts_weight_grad(dy, x, offsets, rows)
    assert torch.equal(y, ns.ns_experts_product(x.contiguous(), w, offsets, rows))
    assert torch.equal(dw, ns.ns_experts_weight_grad(dy, x.contiguous(), offsets, rows))
    sorted_x = x[rows.long()]
    assert torch.equal(y, ns.ns_experts_product(sorted_x, w, offsets))
    assert torch.equal(dw, ns.ns_experts_weight_grad(dy, sorted_x, offsets))


@pytest.mark.parametrize("dtype", DTYPES)
def test_experts_bad_index_data_stays_inside(dtype):
    # row numbers out of range read as zeros; offsets are clamped
    dev = device()
    offsets, rows = routed([40, 90, 20], 50, 88)
    x, w = normal((50, 64), 89, dtype), normal((3, 48, 64), 90, dtype)
    rows[3], rows[60], rows[149] = 50, -1, 2 ** 31 - 1
    y = ns.ns_experts_product(x.to(dev), w.to(dev), offsets.to(dev), rows.to(dev))
    X = np.concatenate([to64(x), np.zeros((1, 64))])
    R = np.where((rows.numpy() < 0) | (rows.numpy() >= 50), 50, rows.numpy())
    W, O = to64(w), offsets.numpy()
    products_near(y, ref.experts_product(X, W, O, R), ref.experts_product(abs(X), abs(W), O, R), 64, dtype)
    dy = normal((150, 48), 91, dtype)
    dw = ns.ns_experts_weight_grad(dy.to(dev), x.to(dev), offsets.to(dev), rows.to(dev))
    D = to64(dy)
    products_near(dw, ref.experts_weight_grad(D, X, O, R), ref.experts_weight_grad(abs(D), abs(X), O, R), 90, dtype)
    rows = rows.clamp(0, 49)
    for bad in ([0, 40, 1000, 150], [-5, 40, 130, 150], [0, 150, 20, 150], [7, 7, 7, 7]):
        o = torch.tensor(bad, dtype=torch.int32)
        out = torch.zeros(150, 48, dtype=dtype, device=dev)
        ns.ns_experts_product(x.to(dev), w.to(dev), o.to(dev), rows.to(dev), y=out)
        assert torch.isfinite(out).all()
        assert torch.isfinite(ns.ns_experts_input_grad(dy.to(dev), w.to(dev), o.to(dev), dx=torch.zeros(
            150, 64, dtype=dtype, device=dev))).all()
        assert torch.isfinite(ns.ns_experts_weight_grad(dy.to(dev), x.to(dev), o.to(dev), rows.to(dev))).all()


def test_experts_unnamed_rows_are_left_alone():
    dev = device()
    offsets = torch.tensor([0, 30, 30, 77], dtype=torch.int32, device=dev)
    x, w = normal((100, 40), 92).to(dev), normal((3, 24, 40), 93).to(dev)
    y = torch.full((100, 24), 7.0, device=dev)
    ns.ns_experts_product(x, w, offsets, y=y)
    assert (y[77:] == 7.0).all() and (y[:77] != 7.0).all()


def test_experts_nan_stays_in_its_rows():
    dev = device()
    offsets, rows = routed([100, 60], 160, 94)
    x, w = normal((160, 64), 95, torch.bfloat16).to(dev), normal((2, 64, 64), 96, torch.bfloat16).to(dev)
    rows = torch.arange(160, dtype=torch.int32)
    x[5] = float("nan")
    w[1, 3] = float("inf")
    y = ns.ns_experts_product(x, w, offsets.to(dev), rows.to(dev))
    assert torch.isnan(y[5]).all()
    ok = torch.isfinite(y)
    ok[5] = True
    assert ok[:100].all() and ok[100:, :3].all() and ok[100:, 4:].all() and not ok[100:, 3].any()


def test_experts_no_rows():
    dev = device()
    o = torch.zeros(4, dtype=torch.int32, device=dev)
    w = torch.ones(3, 16, 24, device=dev)
    none = torch.empty(0, dtype=torch.int32, device=dev)
    assert ns.ns_experts_product(torch.ones(5, 24, device=dev), w, o, none).shape == (0, 16)
    dy = torch.empty(0, 16, device=dev)
    assert ns.ns_experts_input_grad(dy, w, o).shape == (0, 24)
    assert (ns.ns_experts_weight_grad(dy, torch.ones(5, 24, device=dev), o, none) == 0).all()


# ---------------------------------------------------------------- combine

COMBINES = [(1, 1, 8), (1, 8, 2048), (33, 3, 40), (100, 8, 520), (9, 20, 2056), (257, 2, 24), (5, 9, 4104)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", COMBINES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(dtype, case, weighted):
    T, k, C = case
    g = torch.Generator("cpu").manual_seed(100)
    slots = torch.randperm(T * k, generator=g).int().reshape(T, k)
    y, w = normal((T * k, C), 101, dtype), normal((T, k), 102) if weighted else None
    dev = device()
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    S, Y, W = slots.numpy(), to64(y), to64(w) if weighted else None
    got = ns.ns_experts_combine(to(y), to(slots), to(w))
    h = half_step(dtype)
    want, mag = ref.combine(Y, S, W), ref.combine(abs(Y), S, abs(W) if weighted else None)
    near(got, want, h * np.abs(want) + (1 + h) * k * U * mag)
    dout = normal((T, C), 103, dtype)
    dy, dw = ns.ns_experts_combine_backward(to(dout), to(y), to(slots), to(w))
    wy, ww = ref.combine_backward(to64(dout), Y, S, W)
    near(dy, wy, (h + 2 * U) * np.abs(wy))
    if weighted:
        near(dw, ww, C * U * ref.combine_backward(abs(to64(dout)), abs(Y), S, W)[1])
    else:
        assert dw is None


def test_combine_more_tokens_than_a_launch_holds_blocks():
    # 2^24 + 5 tokens: output offsets past 2^32 elements, and blocks that go round
    T, cols, dev = (1 << 24) + 5, 520, device()
    y = normal((16, cols), 105, torch.bfloat16).to(dev)
    slots = (torch.arange(T, device=dev, dtype=torch.int32) % 16).view(T, 1)
    out = ns.ns_experts_combine(y, slots)
    at = torch.cat([torch.arange(0, T, 65537), torch.arange(T - 40, T)]).to(dev)
    assert torch.equal(out[at], y[at % 16])
    w = torch.ones(T, 1, device=dev)
    dw = torch.empty_like(w)
    status = ns.lib().ns_experts_combine_backward(  # no dy: choices share rows of y
        out.data_ptr(), y.data_ptr(), slots.data_ptr(), w.data_ptr(), None, dw.data_ptr(), T, 1, 16, cols,
        ns.NS_DTYPE_BF16, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    norms = (y.double() ** 2).sum(1)
    near(dw[at, 0], to64(norms[at % 16]), to64(norms[at % 16]) * cols * U)


def test_combine_bad_slots_add_nothing():
    dev = device()
    y, w = normal((12, 64), 104), normal((4, 3), 105)
    slots = torch.arange(12, dtype=torch.int32).reshape(4, 3)
    slots[0, 1], slots[2, 0], slots[3, :] = 12, -1, 2 ** 31 - 1
    out = ns.ns_experts_combine(y.to(dev), slots.to(dev), w.to(dev))
    S = slots.numpy()
    near(out, ref.combine(to64(y), S, to64(w)), 3 * U * ref.combine(abs(to64(y)), S, abs(to64(w))) + 1e-38)
    assert (out[3] == 0).all()
    dy, dw = ns.ns_experts_combine_backward(out, y.to(dev), slots.to(dev), w.to(dev), dy=torch.zeros(12, 64, device=dev))
    assert dw[0, 1] == 0 and dw[2, 0] == 0 and (dw[3] == 0).all() and (dy[9:] == 0).all()


# --------------------------------------------- outputs beyond the L2 (32 MiB)


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_of_many_rows_is_that_of_few(dtype):
    dev = device()
    x, dy = normal((5003, 4104), 140, dtype).to(dev), normal((5003, 4104), 141, dtype).to(dev)
    w, b = normal((4104,), 142).to(dev), normal((4104,), 143).to(dev)
    y, mean, rstd = ns.ns_layer_norm(x, w, b)
    dx, dw, db = ns.ns_layer_norm_backward(dy, x, w, mean, rstd)
    assert y.numel() * y.element_size() > 32 << 20
    for i in range(0, 5003, 1000):
        s = slice(i, i + 1000)
        ys, ms, rs = ns.ns_layer_norm(x[s], w, b)
        assert torch.equal(ys, y[s]) and torch.equal(ms, mean[s]) and torch.equal(rs, rstd[s])
        assert torch.equal(ns.ns_layer_norm_backward(dy[s], x[s], w, ms, rs)[0], dx[s])
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    terms = dy.double() * xh
    # xh is off by 3 U of itself and of mean rstd; a sum of 5003 terms
    near(dw, to64(terms.sum(0)), 5100 * U * to64((terms.abs() + dy.double().abs()).sum(0)))
    near(db, to64(dy.double().sum(0)), 5100 * U * to64(dy.double().abs().sum(0)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_experts_products_of_many_rows(dtype):
    dev = device()
    counts, N, K = [4000, 0, 33, 5100, 1], 2056, 1992
    offsets, rows = routed(counts, 3000, 144)
    x, w = normal((3000, K), 145, dtype).to(dev), normal((5, N, K), 146, dtype).to(dev)
    dy = normal((sum(counts), N), 147, dtype).to(dev)
    y = ns.ns_experts_product(x, w, offsets.to(dev), rows.to(dev))
    dx = ns.ns_experts_input_grad(dy, w, offsets.to(dev))
    assert dx.numel() * dx.element_size() > 32 << 20
    for e, c in enumerate(counts):  # (in 64 bits, on the GPU)
        s = slice(int(offsets[e]), int(offsets[e]) + c)
        X, W, D = x[rows[s].to(dev).long()].double(), w[e].double(), dy[s].double()
        products_near(y[s], to64(X @ W.t()), to64(X.abs() @ W.abs().t()), K, dtype)
        products_near(dx[s], to64(D @ W), to64(D.abs() @ W.abs()), N, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_experts_few_rows_of_many_weights(dtype):
    dev = device()
    counts, N, K = ([3, 0, 40, 1, 2, 0, 9, 1] * 9), 520, 520
    M, E = sum(counts), len(counts)
    offsets, rows = routed(counts, 50, 148)
    x, w, dy = normal((50, K), 149, dtype), normal((E, N, K), 150, dtype), normal((M, N), 151, dtype)
    assert w.numel() * w.element_size() > 32 << 20
    X, W, D, R, O = to64(x), to64(w), to64(dy), rows.numpy(), offsets.numpy()
    y = ns.ns_experts_product(x.to(dev), w.to(dev), offsets.to(dev), rows.to(dev))
    assert "tile=32x64" in ns.ns_query_last_config()
    products_near(y, ref.experts_product(X, W, O, R), ref.experts_product(abs(X), abs(W), O, R), K, dtype)
    dx = ns.ns_experts_input_grad(dy.to(dev), w.to(dev), offsets.to(dev))
    products_near(dx, ref.experts_input_grad(D, W, O), ref.experts_input_grad(abs(D), abs(W), O), N, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_backward_of_many_rows(dtype):
    dev = device()
    T, k, cols = 3001, 3, 2056
    slots = torch.randperm(T * k, generator=torch.Generator().manual_seed(152)).int().view(T, k).to(dev)
    y, dout, w = normal((T * k, cols), 153, dtype).to(dev), normal((T, cols), 154, dtype).to(dev), normal((T, k), 155).to(dev)
    dy, dw = ns.ns_experts_combine_backward(dout, y, slots, w)
    assert dy.numel() * dy.element_size() > 32 << 20
    assert torch.equal(dy[slots.long()], (w[:, :, None] * dout.float()[:, None]).to(dtype))  # one product, rounded
    terms = dout.double()[:, None] * y[slots.long()].double()
    near(dw, to64(terms.sum(2)), cols * U * to64(terms.abs().sum(2)))


# ------------------------------------------------------- streams, graphs


def sublayer_step(x, gamma, logit_w, w1, w2, dout, top_k=4):
    """Forward and backward of norm, route, two products with a squared ReLU between, combine."""
    h, mean, rstd = ns.ns_layer_norm(x, gamma)
    logits = h.float() @ logit_w
    r = ns.ns_route(logits, top_k)
    a = ns.ns_experts_product(h, w1, r.offsets, r.rows)
    z = torch.relu(a)
    y = ns.ns_experts_product(z * z, w2, r.offsets)
    out = ns.ns_experts_combine(y, r.slots, r.weights)
    dy, dweights = ns.ns_experts_combine_backward(dout, y, r.slots, r.weights)
    dw2 = ns.ns_experts_weight_grad(dy, z * z, r.offsets)
    da = ns.ns_experts_input_grad(dy, w2, r.offsets) * 2 * z
    dw1 = ns.ns_experts_weight_grad(da, h, r.offsets, r.rows)
    dh = ns.ns_experts_combine(ns.ns_experts_input_grad(da, w1, r.offsets), r.slots)
    dlogits = ns.ns_route_backward(logits, r.ids, dweights)
    dh = dh + (dlogits @ logit_w.t()).to(dh.dtype)
    dx, dgamma, _ = ns.ns_layer_norm_backward(dh, x, gamma, mean, rstd)
    return [out, dw1, dw2, dx, dgamma, dlogits, *ns.orthogonalize_grouped([dw1, dw2])]


def step_inputs(dtype, tokens=200, K=136, N=72, E=12):
    dev = device()
    return (normal((tokens, K), 110, dtype).to(dev), normal((K,), 111, scale=0.1, shift=1.0).to(dev),
            normal((K, E), 112, scale=0.2).to(dev), normal((E, N, K), 113, dtype, 0.1).to(dev),
            normal((E, K, N), 114, dtype, 0.1).to(dev), normal((tokens, K), 115, dtype).to(dev))


@pytest.mark.parametrize("dtype", DTYPES)
def test_step_on_another_stream_and_with_a_poisoned_workspace(dtype):
    args = step_inputs(dtype)
    want = sublayer_step(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = sublayer_step(*args)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ns.ns_set_workspace_poison(1)
    try:
        got = sublayer_step(*args)
    finally:
        ns.ns_set_workspace_poison(0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_operators_captured_into_a_graph():
    # replays with new inputs, eager work and synchronisation between them
    args = step_inputs(torch.bfloat16)
    x, gamma, logit_w, w1, w2, dout = args
    logits = normal((200, 12), 116).to(x.device)

    def ops():
        h, mean, rstd = ns.ns_layer_norm(x, gamma)
        r = ns.ns_route(logits, 4, score="sigmoid")
        y = ns.ns_experts_product(h, w1, r.offsets, r.rows)
        out = ns.ns_experts_combine(y, r.slots, r.weights)
        dy, dwt = ns.ns_experts_combine_backward(out, y, r.slots, r.weights)
        dw1 = ns.ns_experts_weight_grad(dy, h, r.offsets, r.rows)
        dh = ns.ns_experts_combine(ns.ns_experts_input_grad(dy, w1, r.offsets), r.slots)
        dl = ns.ns_route_backward(logits, r.ids, dwt, score="sigmoid")
        return [h, r.ids, r.weights, r.offsets, r.rows, r.slots, y, out, dy, dwt, dw1, dh, dl,
                *ns.ns_layer_norm_backward(dh, x, gamma, mean, rstd)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops()
        side.synchronize()
        allocations = ns.ns_workspace_allocations()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = ops()
    torch.cuda.synchronize()
    assert ns.ns_workspace_allocations() == allocations
    for i in range(4):
        x.copy_(normal((200, 136), 120 + i, torch.bfloat16))
        logits.copy_(normal((200, 12), 130 + i))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ops()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


def test_what_ran_is_named():
    dev = device()
    x = torch.randn(4, 64, device=dev)
    ns.ns_layer_norm(x)
    assert ns.ns_query_last_config().startswith("layer norm")
    r = ns.ns_route(x, 2)
    assert ns.ns_query_last_config().startswith("route")
    ns.ns_experts_product(x, torch.randn(64, 8, 64, device=dev), r.offsets, r.rows)
    assert ns.ns_query_last_config().startswith("experts product")
    ns.ns_timing_reset()
    ns.ns_timing_enable(1 << ns.NS_KIND_ROUTE)
    try:
        ns.ns_route(x, 2)
        assert ns.ns_timing_query(ns.NS_KIND_ROUTE)[1] == 1
    finally:
        ns.ns_timing_enable(0)
        ns.ns_timing_reset()


def test_example_learns_and_decodes():
    import importlib.util
    import pathlib
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "moe_sublayer.py"
    spec = importlib.util.spec_from_file_location("moe_sublayer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    device()
    losses, worst = example.main(["--tokens", "520", "--width", "136", "--hidden", "72", "--experts", "12", "--steps", "25"])
    assert all(np.isfinite(losses)) and losses[-1] < 0.9 * losses[0]
    assert worst == 0.0  # the same kernels on the same values
