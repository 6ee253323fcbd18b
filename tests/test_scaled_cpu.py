"""The sublayer in 8 bits without a GPU: the oracle against closed forms and differences, and the entry points' refusals,
which come before the device is touched."""

import ctypes

import numpy as np
import pytest
import torch

import newton_schulz_07_amd as ns
from oracle import scaled as ref
from tests.test_sublayer_cpu import A, B, BIG, C, D, F, differences, status

FAR = 1 << 40


@pytest.fixture
def rng():
    return np.random.default_rng(11)


def test_the_oracles_values_are_torchs():
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, ref.E4M3, equal_nan=True)


def test_the_oracles_rounding_is_torchs(rng):
    v = np.concatenate([rng.normal(size=4000) * np.exp(3 * rng.normal(size=4000)), ref.POSITIVE,
                        (ref.POSITIVE[1:] + ref.POSITIVE[:-1]) / 2, [0.0, -0.0, 2.0 ** -10, -(2.0 ** -11)]])
    v = v[np.abs(v) <= 448].astype(np.float32)
    got = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, ref.codes(v))


def test_the_scale_is_the_least_that_is_enough():
    for top, byte in ((448.0, 127), (448.5, 128), (224.0, 126), (225.0, 127), (0.0, 1), (1e-40, 1),
                      (448 * 2.0 ** -126, 1), (449 * 2.0 ** -126, 2), (float(np.finfo(np.float32).max), 247)):
        assert ref.scale_of(np.array([top, -top / 2, np.nan, np.inf])) == byte, top


def test_rms_norm_gradient(rng):
    t, w, dy, dt = rng.normal(size=(5, 12)), rng.normal(size=12), rng.normal(size=(5, 12)), rng.normal(size=(5, 12))
    dx, dw = ref.rms_norm_backward(dy, t, w, ref.rms_norm(t, w)[1], dt)
    for grad, at, f in ((dx, t, lambda v: (dy * ref.rms_norm(v, w)[0]).sum() + (dt * v).sum()),
                        (dw, w, lambda v: (dy * ref.rms_norm(t, v)[0]).sum())):
        d = rng.normal(size=at.shape)
        assert abs((grad * d).sum() - differences(f, at, d)) < 1e-7


# -------------------------------------------------------------- refusals

E, G = (0x10000000 * i for i in range(6, 8))
NORM = dict(x=A, ldx=64, residual=B, ldr=64, weight=C, total=D, y=E, q=F, scales=F + 65536, rstd=G, rows=10, cols=64,
            dtype=1, param_dtype=0, eps=1e-6, stream=None)
NORM_BACK = dict(dy=A, lddy=64, x=B, ldx=64, weight=C, rstd=C + 4096, dtotal=D, lddt=64, dx=E, dweight=F, rows=10,
                 cols=64, dtype=1, param_dtype=0, stream=None)
ROWS = dict(x=A, ldx=64, q=B, scales=C, rows=10, cols=64, dtype=1, stream=None)
WEIGHTS = dict(w=A, q=B, scales=C, qt=D, scales_t=E, experts=3, fan_out=32, fan_in=64, dtype=1, stream=None)
BACK = dict(q=A, scales=B, x=C, matrices=3, rows=32, cols=64, block_rows=128, dtype=1, stream=None)
PRODUCT = dict(x=A, x_scales=A + 65537, n_x=20, rows=B, w=C, w_scales=C + 65537, offsets=D, y=E, n_rows=30, experts=4,
               fan_out=32, fan_in=64, dtype=1, stream=None)
GRAD = dict(dy=A, x=B, x_scales=B + 65537, n_x=20, rows=C, offsets=C + 65536, dw=D, n_rows=30, experts=4, fan_out=32,
            fan_in=64, dtype=1, stream=None)
ALL = [("ns_rms_norm", NORM), ("ns_rms_norm_backward", NORM_BACK), ("ns_quantize", ROWS),
       ("ns_quantize_weights", WEIGHTS), ("ns_dequantize", BACK), ("ns_experts_product_scaled", PRODUCT),
       ("ns_experts_weight_grad_scaled", GRAD)]


@pytest.mark.parametrize("name,defaults,changes,want", [
    (n, d, c, s) for n, d, cases in [
        ("ns_rms_norm", NORM, [
            (dict(x=0), 1), (dict(x=A + 8), 3), (dict(residual=0), 1), (dict(total=0), 1), (dict(residual=B + 4), 3),
            (dict(y=0, q=0, scales=0), 1), (dict(q=0), 1), (dict(scales=0), 1), (dict(y=E + 2), 3), (dict(q=F + 8), 3),
            (dict(weight=C + 4), 3), (dict(rstd=G + 2), 3), (dict(rows=-1), 1), (dict(rows=BIG), 1), (dict(cols=0), 1),
            (dict(cols=(1 << 20) + 16, ldx=(1 << 20) + 16, ldr=(1 << 20) + 16), 1), (dict(ldx=63), 1),
            (dict(ldr=63), 1), (dict(ldr=1 << 21), 1), (dict(cols=56), 3), (dict(dtype=2), 2), (dict(param_dtype=7), 2),
            (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(y=A), 1), (dict(total=B), 1), (dict(q=E + 16), 1),
            (dict(scales=F + 16), 1), (dict(rstd=D), 1)]),
        ("ns_rms_norm_backward", NORM_BACK, [
            (dict(dy=0), 1), (dict(x=0), 1), (dict(rstd=0), 1), (dict(dx=A), 1), (dict(dx=B + 16), 1), (dict(dx=D), 1),
            (dict(dx=E + 4), 3), (dict(dweight=E), 1), (dict(dtotal=D + 8), 3), (dict(lddy=60), 1), (dict(lddt=60), 1),
            (dict(dtype=7), 2), (dict(param_dtype=2), 2), (dict(rows=-3), 1), (dict(cols=0), 1)]),
        ("ns_quantize", ROWS, [
            (dict(x=0), 1), (dict(q=0), 1), (dict(scales=0), 1), (dict(x=A + 8), 3), (dict(q=B + 8), 3),
            (dict(cols=72, ldx=72), 3), (dict(cols=0), 1), (dict(ldx=48), 1), (dict(rows=-1), 1), (dict(rows=BIG), 1),
            (dict(rows=1 << 30, cols=512, ldx=512, q=FAR, scales=2 * FAR), 1), (dict(dtype=2), 2), (dict(q=A), 1),
            (dict(scales=B + 100), 1)]),
        ("ns_quantize_weights", WEIGHTS, [
            (dict(w=0), 1), (dict(q=0), 1), (dict(scales=0), 1), (dict(qt=0), 1), (dict(scales_t=0), 1),
            (dict(w=A + 8), 3), (dict(qt=D + 8), 3), (dict(fan_out=24), 3), (dict(fan_in=72), 3), (dict(experts=0), 1),
            (dict(experts=1025), 1), (dict(fan_out=1 << 15, fan_in=1 << 14), 1),
            (dict(experts=1024, fan_out=1 << 14, fan_in=1 << 14), 1), (dict(dtype=2), 2), (dict(q=A), 1),
            (dict(qt=B), 1), (dict(scales_t=D + 5), 1)]),
        ("ns_dequantize", BACK, [
            (dict(q=0), 1), (dict(scales=0), 1), (dict(x=0), 1), (dict(q=A + 8), 3), (dict(x=C + 4), 3),
            (dict(block_rows=64), 1), (dict(matrices=-1), 1), (dict(rows=-1), 1), (dict(matrices=1 << 20, rows=1 << 11), 1),
            (dict(cols=24), 3), (dict(dtype=2), 2), (dict(x=A), 1), (dict(scales=C + 5), 1)]),
        ("ns_experts_product_scaled", PRODUCT, [
            (dict(x=0), 1), (dict(x_scales=0), 1), (dict(w=0), 1), (dict(w_scales=0), 1), (dict(offsets=0), 1),
            (dict(y=0), 1), (dict(rows=0), 1), (dict(n_x=0), 1), (dict(fan_out=40), 3), (dict(fan_in=72), 3),
            (dict(experts=0), 1), (dict(experts=1025), 1), (dict(n_rows=-1), 1), (dict(n_rows=BIG - 1023), 1),
            (dict(fan_out=1 << 15, fan_in=1 << 14), 1), (dict(n_x=1 << 25), 1), (dict(dtype=2), 2), (dict(y=A), 1),
            (dict(y=C + 16), 1), (dict(x=A + 8), 3), (dict(rows=B + 2), 3), (dict(offsets=D + 1), 3)]),
        ("ns_experts_weight_grad_scaled", GRAD, [
            (dict(dy=0), 1), (dict(x=0), 1), (dict(x_scales=0), 1), (dict(offsets=0), 1), (dict(dw=0), 1),
            (dict(dw=A), 1), (dict(dw=B), 1), (dict(rows=0), 1), (dict(n_x=0), 1), (dict(fan_out=8), 3),
            (dict(dtype=2), 2), (dict(n_x=1 << 24), 1), (dict(n_rows=BIG - 1023), 1)]),
    ] for c, s in cases])
def test_refusals(name, defaults, changes, want):
    assert status(name, defaults, changes) == want


@pytest.mark.parametrize("name,defaults,changes", [
    *((n, d, {}) for n, d in ALL), ("ns_rms_norm", NORM, dict(residual=0, total=0, weight=0, y=0)),
    ("ns_rms_norm", NORM, dict(cols=57, q=0, scales=0)), ("ns_rms_norm_backward", NORM_BACK, dict(dtotal=0, dx=0)),
    ("ns_rms_norm_backward", NORM_BACK, dict(rows=0, dy=0, x=0, rstd=0, dtotal=0)),
    ("ns_quantize_weights", WEIGHTS, dict(qt=0, scales_t=0)), ("ns_dequantize", BACK, dict(block_rows=1)),
    ("ns_experts_product_scaled", PRODUCT, dict(experts=1, offsets=0, rows=0, n_x=30)),
    ("ns_experts_weight_grad_scaled", GRAD, dict(n_rows=0, rows=0, x=0, x_scales=0, dy=0))])
@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only where there is no device")
def test_good_arguments_get_as_far_as_the_device(name, defaults, changes):
    assert status(name, defaults, changes) not in (0, 1, 2, 3), ns.lib().ns_last_error().decode()


@pytest.mark.parametrize("name,defaults,changes", [
    ("ns_rms_norm", NORM, dict(rows=0)), ("ns_rms_norm_backward", NORM_BACK, dict(rows=0, dweight=0)),
    ("ns_rms_norm_backward", NORM_BACK, dict(dx=0, dweight=0)), ("ns_quantize", ROWS, dict(rows=0)),
    ("ns_dequantize", BACK, dict(matrices=0)), ("ns_dequantize", BACK, dict(rows=0)),
    ("ns_experts_product_scaled", PRODUCT, dict(n_rows=0))])
def test_nothing_to_do(name, defaults, changes):
    assert status(name, defaults, changes) == 0


def test_signatures_cover_every_argument():
    for name, defaults in ALL:
        assert len(ns.SIGNATURES[name][1]) == len(defaults)
        assert ns.SIGNATURES[name][1][-1] is ctypes.c_void_p


def test_binding_refuses_host_tensors():
    x, s = torch.zeros(4, 64), torch.zeros(4, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    q, o = x.to(torch.float8_e4m3fn), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: ns.ns_rms_norm(x), lambda: ns.ns_rms_norm_backward(x, x, None, x),
                 lambda: ns.ns_quantize(x), lambda: ns.ns_quantize_weights(x), lambda: ns.ns_dequantize(q, s),
                 lambda: ns.ns_experts_product_scaled(q, s, q, s),
                 lambda: ns.ns_experts_weight_grad_scaled(x, q, s, o)):
        with pytest.raises(ValueError):
            call()


def test_every_operators_name_is_the_packages():
    for name in ("ns_rms_norm", "ns_quantize", "ns_experts_product_scaled", "Scaled", "ns_route"):
        assert name in dir(ns) and getattr(ns, name) is not None
    with pytest.raises(AttributeError):
        ns.ns_nothing
