"""The mixture-of-experts sublayer without a GPU: the oracle's gradients against differences, and the entry points'
refusals, which come before the device is touched."""

import ctypes

import numpy as np
import pytest
import torch

import newton_schulz_07_amd as ns
from oracle import sublayer as ref

A, B, C, D, F = (0x10000000 * i for i in range(1, 6))  # far apart, 16-byte aligned


def differences(f, x, d, h=1e-5):
    """Directional derivative of f at x along d."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.fixture
def rng():
    return np.random.default_rng(7)


def test_layer_norm_gradient(rng):
    x, w, b, dy = rng.normal(size=(5, 12)), rng.normal(size=12), rng.normal(size=12), rng.normal(size=(5, 12))
    _, mean, rstd = ref.layer_norm(x, w, b)
    dx, dw, db = ref.layer_norm_backward(dy, x, w, mean, rstd)
    for grad, at, f in ((dx, x, lambda v: (dy * ref.layer_norm(v, w, b)[0]).sum()),
                        (dw, w, lambda v: (dy * ref.layer_norm(x, v, b)[0]).sum()),
                        (db, b, lambda v: (dy * ref.layer_norm(x, w, v)[0]).sum())):
        d = rng.normal(size=at.shape)
        assert abs((grad * d).sum() - differences(f, at, d)) < 1e-7


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient(rng, score, renorm):
    z, dw = rng.normal(size=(6, 10)), rng.normal(size=(6, 3))
    kw = dict(score=score, renormalize=renorm, scale=1.7)
    ids = ref.route(z, 3, **kw)[0]
    d = rng.normal(size=z.shape)
    got = (ref.route_backward(z, ids, dw, **kw) * d).sum()

    def loss(v):
        s = np.take_along_axis(ref.scores(v, score), ids, 1)
        return (dw * 1.7 * (s / s.sum(1, keepdims=True) if renorm else s)).sum()
    assert abs(got - differences(loss, z, d)) < 1e-8


def test_experts_and_combine_gradients(rng):
    offsets, rows = np.array([0, 3, 3, 8]), np.array([0, 2, 1, 3, 0, 1, 2, 3])
    x, w = rng.normal(size=(4, 6)), rng.normal(size=(3, 5, 6))
    slots, wt = rng.permutation(8).reshape(4, 2), rng.normal(size=(4, 2))
    dout = rng.normal(size=(4, 5))

    def loss(x, w, wt):
        return (dout * ref.combine(ref.experts_product(x, w, offsets, rows), slots, wt)).sum()
    y = ref.experts_product(x, w, offsets, rows)
    dy, dwt = ref.combine_backward(dout, y, slots, wt)
    dw = ref.experts_weight_grad(dy, x, offsets, rows)
    dxs = ref.experts_input_grad(dy, w, offsets)
    dx = np.zeros_like(x)
    np.add.at(dx, rows, dxs)
    for grad, at, f in ((dx, x, lambda v: loss(v, w, wt)), (dw, w, lambda v: loss(x, v, wt)),
                        (dwt, wt, lambda v: loss(x, w, v))):
        d = rng.normal(size=at.shape)
        assert abs((grad * d).sum() - differences(f, at, d)) < 1e-8


# -------------------------------------------------------------- refusals


def status(name, defaults, changes):
    args = list({**defaults, **changes}.values())
    st = getattr(ns.lib(), name)(*args)
    if st in (1, 2, 3):
        assert ns.lib().ns_last_error().decode() != ""
    return st


NORM = dict(x=A, ldx=64, weight=B, bias=B + 4096, y=C, mean=D, rstd=D + 65536, rows=10, cols=64, dtype=1, param_dtype=0,
            eps=1e-5, stream=None)
NORM_BACK = dict(dy=A, lddy=64, x=B, ldx=64, weight=C, mean=C + 4096, rstd=C + 8192, dx=D, dweight=F, dbias=F + 4096,
                 rows=10, cols=64, dtype=1, param_dtype=0, stream=None)
ROUTE = dict(logits=A, ld=64, bias=B, ids=C, weights=C + 65536, offsets=D, rows=D + 65536, slots=D + 131072, tokens=10,
             experts=64, top_k=4, groups=8, top_groups=2, group_best=2, score=0, renormalize=1, scale=1.0, dtype=0,
             stream=None)
ROUTE_BACK = dict(logits=A, ld=64, ids=B, dweights=C, dlogits=D, tokens=10, experts=64, top_k=4, score=0, renormalize=1,
                  scale=1.0, dtype=0, stream=None)
PRODUCT = dict(x=A, ldx=64, n_x=20, rows=B, w=C, offsets=B + 65536, y=D, n_rows=30, experts=4, fan_out=32, fan_in=64,
               dtype=1, stream=None)
INPUT = dict(dy=A, w=C, offsets=B, dx=D, n_rows=30, experts=4, fan_out=32, fan_in=64, dtype=1, stream=None)
WEIGHT = dict(dy=A, x=F, ldx=64, n_x=20, rows=B, offsets=B + 65536, dw=D, n_rows=30, experts=4, fan_out=32, fan_in=64,
              dtype=1, stream=None)
COMBINE = dict(y=A, slots=B, weights=C, out=D, tokens=10, top_k=2, n_rows=20, cols=64, dtype=1, stream=None)
COMBINE_BACK = dict(dout=A, y=B, slots=C, weights=C + 65536, dy=D, dweights=F, tokens=10, top_k=2, n_rows=20, cols=64,
                    dtype=1, stream=None)

BIG = 1 << 31


@pytest.mark.parametrize("name,defaults,changes,want", [
    (n, d, c, s) for n, d, cases in [
        ("ns_layer_norm", NORM, [
            (dict(x=0), 1), (dict(y=0), 1), (dict(x=A + 8), 3), (dict(y=C + 2), 3), (dict(weight=B + 4), 3),
            (dict(mean=D + 2), 3), (dict(rows=-1), 1), (dict(rows=BIG), 1), (dict(cols=0), 1),
            (dict(cols=(1 << 20) + 8, ldx=(1 << 20) + 8), 1), (dict(ldx=63), 1), (dict(ldx=1 << 21), 1),
            (dict(dtype=2), 2), (dict(param_dtype=-1), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
            (dict(y=A), 1), (dict(mean=C + 64), 1), (dict(mean=D, rstd=D), 1)]),
        ("ns_layer_norm_backward", NORM_BACK, [
            (dict(dy=0), 1), (dict(x=0), 1), (dict(mean=0), 1), (dict(rstd=0), 1), (dict(dx=A), 1), (dict(dx=B), 1),
            (dict(dx=D + 4), 3), (dict(dweight=F, dbias=F), 1), (dict(lddy=60), 1), (dict(dtype=7), 2),
            (dict(rows=-3), 1)]),
        ("ns_route", ROUTE, [
            (dict(logits=0), 1), (dict(ids=0), 1), (dict(weights=0), 1), (dict(offsets=0), 1), (dict(rows=0), 1),
            (dict(logits=A + 4), 3), (dict(ids=C + 2), 3), (dict(experts=0), 1), (dict(experts=1025, ld=1025), 1),
            (dict(top_k=0), 1), (dict(top_k=65), 1), (dict(experts=3, top_k=4, groups=1), 1), (dict(groups=0), 1),
            (dict(groups=7), 1), (dict(top_groups=9), 1), (dict(top_groups=0), 1),
            (dict(top_k=9, top_groups=1), 1), (dict(group_best=3), 1), (dict(score=2), 1), (dict(ld=63), 1),
            (dict(tokens=-1), 1), (dict(tokens=BIG // 4, top_k=4), 1), (dict(dtype=3), 2), (dict(ids=A), 1),
            (dict(slots=D + 65536), 1), (dict(tokens=1 << 25, top_k=1), 1)]),
        ("ns_route_backward", ROUTE_BACK, [
            (dict(logits=0), 1), (dict(ids=0), 1), (dict(dweights=0), 1), (dict(dlogits=0), 1), (dict(dlogits=A), 1),
            (dict(top_k=65), 1), (dict(score=-1), 1), (dict(dtype=2), 2), (dict(dlogits=D + 8), 3),
            (dict(tokens=1 << 25), 1)]),
        ("ns_experts_product", PRODUCT, [
            (dict(x=0), 1), (dict(w=0), 1), (dict(offsets=0), 1), (dict(y=0), 1), (dict(rows=0), 1),
            (dict(n_x=0), 1), (dict(fan_out=36), 3), (dict(fan_in=60), 3), (dict(ldx=68), 3), (dict(ldx=56), 1),
            (dict(experts=0), 1), (dict(experts=1025), 1), (dict(n_rows=-1), 1), (dict(fan_out=0), 1),
            (dict(fan_out=1 << 16, fan_in=1 << 16, ldx=1 << 16), 1), (dict(n_x=1 << 25), 1), (dict(dtype=2), 2),
            (dict(y=A), 1), (dict(y=C + 16), 1), (dict(x=A + 8), 3), (dict(rows=B + 2), 3)]),
        ("ns_experts_input_grad", INPUT, [
            (dict(dy=0), 1), (dict(w=0), 1), (dict(offsets=0), 1), (dict(dx=0), 1), (dict(dx=A), 1),
            (dict(fan_in=12), 3), (dict(dtype=2), 2), (dict(n_rows=BIG), 1)]),
        ("ns_experts_weight_grad", WEIGHT, [
            (dict(dy=0), 1), (dict(x=0), 1), (dict(offsets=0), 1), (dict(dw=0), 1), (dict(dw=A), 1), (dict(dw=F), 1),
            (dict(rows=0), 1), (dict(n_x=0), 1), (dict(fan_out=9), 3), (dict(dtype=2), 2), (dict(ldx=1 << 21), 1)]),
        ("ns_experts_combine", COMBINE, [
            (dict(y=0), 1), (dict(slots=0), 1), (dict(out=0), 1), (dict(out=A), 1), (dict(cols=60), 3),
            (dict(top_k=0), 1), (dict(cols=0), 1), (dict(tokens=BIG), 1), (dict(dtype=2), 2), (dict(slots=B + 1), 3)]),
        ("ns_experts_combine_backward", COMBINE_BACK, [
            (dict(dout=0), 1), (dict(y=0), 1), (dict(slots=0), 1), (dict(dy=A), 1), (dict(dy=B), 1), (dict(cols=4), 3),
            (dict(dweights=C), 1), (dict(top_k=0), 1), (dict(dtype=2), 2)]),
    ] for c, s in cases])
def test_refusals(name, defaults, changes, want):
    assert status(name, defaults, changes) == want


@pytest.mark.parametrize("name,defaults", [
    ("ns_layer_norm", NORM), ("ns_layer_norm_backward", NORM_BACK), ("ns_route", ROUTE),
    ("ns_route_backward", ROUTE_BACK), ("ns_experts_product", PRODUCT), ("ns_experts_input_grad", INPUT),
    ("ns_experts_weight_grad", WEIGHT), ("ns_experts_combine", COMBINE),
    ("ns_experts_combine_backward", COMBINE_BACK)])
@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only where there is no device")
def test_good_arguments_get_as_far_as_the_device(name, defaults):
    assert status(name, defaults, {}) not in (0, 1, 2, 3), ns.lib().ns_last_error().decode()


@pytest.mark.parametrize("name,defaults,changes", [
    ("ns_layer_norm", NORM, dict(rows=0)), ("ns_route_backward", ROUTE_BACK, dict(tokens=0)),
    ("ns_experts_product", PRODUCT, dict(n_rows=0)), ("ns_experts_input_grad", INPUT, dict(n_rows=0)),
    ("ns_experts_combine", COMBINE, dict(tokens=0)), ("ns_experts_combine_backward", COMBINE_BACK, dict(tokens=0))])
def test_nothing_to_do(name, defaults, changes):
    assert status(name, defaults, changes) == 0


def test_binding_refuses_host_tensors_and_other_shapes():
    x, w = torch.zeros(4, 64), torch.zeros(2, 8, 64)
    o, i = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: ns.ns_layer_norm(x), lambda: ns.ns_layer_norm_backward(x, x, None, x, x),
                 lambda: ns.ns_route(x, 2), lambda: ns.ns_route_backward(x, i, x),
                 lambda: ns.ns_experts_product(x, w, o), lambda: ns.ns_experts_input_grad(x, w, o),
                 lambda: ns.ns_experts_weight_grad(x, x, o), lambda: ns.ns_experts_combine(x, i),
                 lambda: ns.ns_experts_combine_backward(x, x, i)):
        with pytest.raises(ValueError):
            call()


def test_signatures_cover_every_argument():
    for name, defaults in (("ns_layer_norm", NORM), ("ns_layer_norm_backward", NORM_BACK), ("ns_route", ROUTE),
                           ("ns_route_backward", ROUTE_BACK), ("ns_experts_product", PRODUCT),
                           ("ns_experts_input_grad", INPUT), ("ns_experts_weight_grad", WEIGHT),
                           ("ns_experts_combine", COMBINE), ("ns_experts_combine_backward", COMBINE_BACK)):
        assert len(ns.SIGNATURES[name][1]) == len(defaults)
        assert ns.SIGNATURES[name][1][-1] is ctypes.c_void_p
