"""Edge cases of the mixture-of-experts sublayer's operators against the oracle in float64: keys that cancel, masked
experts with a bias, saturated scores, rows that nothing names, launches at their largest.

Error bounds as in test_gpu_sublayer.py: U = 2^-24; a store to type T is off by at most half a step.
"""

import numpy as np
import pytest
import torch

import newton_schulz_07_amd as ns
from oracle import sublayer as ref
from tests.gpu_util import device, to64
from tests.test_gpu_sublayer import DTYPES, U, check_route, half_step, near, normal

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------- routing


@pytest.mark.parametrize("tokens", [1500, 4500])  # a wave to a token, and 16 lanes
@pytest.mark.parametrize("score,shift,scale,by", [
    ("softmax", 0.0, 0.5, 256.0), ("softmax", 0.0, 0.5, 1024.0),  # scores of about 2^-7: beside 1024 they keep 6 bits
    ("sigmoid", 0.0, 1.5, 16000.0), ("sigmoid", -10.0, 1.0, 16.0),
])
def test_route_ranks_groups_whose_biases_cancel(tokens, score, shift, scale, by):
    # the two experts of a group have keys near `by` and -`by`: their sum is far below either's rounding; all the
    # experts of the chosen groups are chosen
    logits = normal((tokens, 128), 200, scale=scale, shift=shift)
    bias = torch.tensor([by, -by]).repeat(64)
    kw = dict(groups=64, top_groups=7, group_best=2, score=score)
    r = ns.ns_route(logits.to(device()), 14, bias=bias.to(device()), **kw)
    check_route(logits, (14,), dict(kw, bias=to64(bias)), r)


def test_route_ranks_groups_beside_a_closed_one():
    # a bias that takes a whole group out does not blur the others' ranks
    logits = normal((4500, 64), 201)
    bias = normal((64,), 202, scale=0.1)
    bias[8:16] = -1e9
    kw = dict(groups=8, top_groups=4, group_best=2, score="sigmoid")
    r = ns.ns_route(logits.to(device()), 6, bias=bias.to(device()), **kw)
    check_route(logits, (6,), dict(kw, bias=to64(bias)), r)
    assert not ((r.ids >= 8) & (r.ids < 16)).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("copies", [1, 800])  # a wave to a token, and 16 lanes
def test_route_masked_experts_come_last_with_a_bias(score, dtype, copies):
    inf = float("inf")
    logits = torch.tensor([[0.0, -1.0, -inf, -2.0], [-inf, -inf, 3.0, -inf], [-inf] * 4, [-inf, 1.0, -inf, 1.0],
                           [1.0, -inf, 0.5, 2.0], [-3.0, 0.0, -1.0, -inf]]).to(dtype).repeat(copies, 1)
    bias = torch.tensor([0.0, 0.0, 0.9, 0.0])
    want = torch.tensor([[0, 1, 3, 2], [2, 0, 1, 3], [0, 1, 2, 3], [1, 3, 0, 2], [2, 3, 0, 1], [2, 1, 0, 3]])
    dev = device()
    for k in (1, 2, 4):
        r = ns.ns_route(logits.to(dev), k, bias=bias.to(dev), score=score)
        if score == "sigmoid":  # (softmax scores of the last rows order differently: the oracle's below)
            assert torch.equal(r.ids.cpu().long(), want[:, :k].repeat(copies, 1))
        check_route(logits, (k,), dict(score=score, bias=to64(bias)), r)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_best", [1, 2])
@pytest.mark.parametrize("tokens", [300, 4500])
@pytest.mark.parametrize("experts,groups", [(12, 6), (24, 6), (96, 8)])
def test_route_masked_experts_in_groups_with_a_bias(score, group_best, tokens, experts, groups):
    # masked ones add nothing to a group's rank; a group of nothing else comes last, whatever its biases are
    logits = normal((tokens, experts), 203 + experts)
    gone = torch.rand(tokens, experts, generator=torch.Generator().manual_seed(204)) < 0.5
    gone[::3, :experts // groups] = True
    gone[7::50] = True
    logits[gone] = -float("inf")
    bias = normal((experts,), 205, scale=0.3)
    bias[:experts // groups] = 5.0
    kw = dict(groups=groups, top_groups=groups // 2, group_best=group_best, score=score)
    r = ns.ns_route(logits.to(device()), 4, bias=bias.to(device()), **kw)
    check_route(logits, (4,), dict(kw, bias=to64(bias)), r)
    some = ~gone.view(tokens, groups, -1).all(2)  # groups with an expert left
    best = r.ids[:, 0].cpu().long()
    assert some.gather(1, (best // (experts // groups))[:, None])[some.any(1)].all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_of_saturated_sigmoids(dtype, renorm):
    # 1 - s from the logit: the gradient of the chosen, highest logits keeps its bits
    T, E, k = 130, 40, 6
    logits = normal((T, E), 206, dtype, 1.0)
    for t in range(T):  # logits from 8 to 40 and from -8 to -40 among the others, alone in some rows
        g = torch.Generator().manual_seed(1000 + t)
        far = (8 + 32 * torch.rand(E, generator=g)) * (1 if t % 2 else -1)
        at = torch.randperm(E, generator=g)[:E if t % 5 == 0 else 5]
        logits[t, at] = far[at].to(dtype)
    dev = device()
    ids = ns.ns_route(logits.to(dev), k, score="sigmoid").ids
    d = normal((T, k), 207)
    got = ns.ns_route_backward(logits.to(dev), ids, d.to(dev), score="sigmoid", renormalize=renorm, scale=1.5)
    L, I, D = to64(logits), ids.cpu().numpy(), to64(d)
    s, c = 1 / (1 + np.exp(-L)), 1 / (1 + np.exp(L))
    sj = np.take_along_axis(s, I, 1)
    mag = 1.5 * np.abs(D)
    ds = 1.5 * D
    if renorm:
        tot = sj.sum(1, keepdims=True) + 1e-20
        ds = (ds - (ds * sj).sum(1, keepdims=True) / tot) / tot
        mag = (mag + (mag * sj).sum(1, keepdims=True) / tot) / tot
    want, full = np.zeros_like(s), np.zeros_like(s)
    np.put_along_axis(want, I, ds, 1)
    np.put_along_axis(full, I, mag, 1)
    want, into = want * s * c, full * s * c
    near(to64(torch.from_numpy(ref.route_backward(L, I, D, "sigmoid", renorm, 1.5))), want, 1e-13 * into)
    near(got, want, half_step(dtype) * np.abs(want) + (64 + E / 8) * U * into + 1e-38)


# --------------------------------------------------------------- combine


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [0, 1, 40])
def test_combine_backward_gives_spare_rows_no_gradient(dtype, tokens):
    # more rows of y than choices: the rows that no choice names have a gradient of zero
    dev, rows, cols = device(), 200, 136
    slots = torch.randperm(rows, generator=torch.Generator().manual_seed(208))[:3 * tokens].int().view(tokens, 3)
    y, dout, w = normal((rows, cols), 209, dtype), normal((tokens, cols), 210, dtype), normal((tokens, 3), 211)
    torch.cuda.empty_cache()
    held = torch.full((rows, cols), float("nan"), dtype=dtype, device=dev)  # what a buffer taken next would hold
    del held
    want, _ = ref.combine_backward(to64(dout), to64(y), slots.numpy(), to64(w))
    for weights in (w, None):
        if weights is None:
            want, _ = ref.combine_backward(to64(dout), to64(y), slots.numpy())
        dy, _ = ns.ns_experts_combine_backward(dout.to(dev), y.to(dev), slots.to(dev),
                                               None if weights is None else weights.to(dev))
        near(dy, want, (half_step(dtype) + 2 * U) * np.abs(want))
        held = torch.full_like(dy, float("nan"))
        del held, dy


def test_combine_of_the_most_tokens():
    # 2^31 - 1 tokens: counts of blocks past 32 bits
    T, cols, dev = (1 << 31) - 1, 8, device()
    y = normal((16, cols), 213, torch.bfloat16).to(dev)
    slots = torch.arange(16, device=dev, dtype=torch.int32).repeat(1 << 27)[:T].view(T, 1)
    out = ns.ns_experts_combine(y, slots)
    at = torch.cat([torch.arange(0, T, 16777259), torch.arange(T - 40, T)]).to(dev)
    assert torch.equal(out[at], y[at % 16])
    dw = torch.empty(T, 1, device=dev)
    status = ns.lib().ns_experts_combine_backward(  # no dy: choices share rows of y
        out.data_ptr(), y.data_ptr(), slots.data_ptr(), None, None, dw.data_ptr(), T, 1, 16, cols, ns.NS_DTYPE_BF16,
        torch.cuda.current_stream().cuda_stream)
    assert status == 0
    norms = (y.double() ** 2).sum(1)
    near(dw[at, 0], to64(norms[at % 16]), to64(norms[at % 16]) * cols * U)
    del out, dw, slots
    torch.cuda.empty_cache()
