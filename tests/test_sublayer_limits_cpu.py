"""The largest counts of choices and of experts' rows that the entry points take, without a GPU: the kernels step
through them in 32-bit numbers, up to 1024 of them past the last one."""

import pytest
import torch

from tests.test_sublayer_cpu import INPUT, PRODUCT, ROUTE, WEIGHT, status

MOST = (1 << 31) - 1024

# (made-up addresses, so far apart that no two operands of these sizes meet)
FAR = 1 << 50


def spread(defaults, **changes):
    """defaults with every pointer that is not null moved far from the others, and the changes."""
    pointers = [k for k, v in defaults.items() if isinstance(v, int) and v >= 0x10000000]
    return {**{k: FAR * (i + 1) for i, k in enumerate(pointers)}, **changes}


# where a count is at its limit, and its smallest value past it
LIMITS = [
    ("ns_route", ROUTE, lambda n: dict(tokens=n, top_k=64, groups=1, top_groups=1), MOST // 64),
    ("ns_experts_product", PRODUCT, lambda n: dict(n_rows=n, n_x=n, rows=0, ldx=64), MOST),
    ("ns_experts_input_grad", INPUT, lambda n: dict(n_rows=n), MOST),
    ("ns_experts_weight_grad", WEIGHT, lambda n: dict(n_rows=n, n_x=n, rows=0), MOST),
]


@pytest.mark.parametrize("name,defaults,sized,most", LIMITS)
def test_counts_past_the_limit_are_refused(name, defaults, sized, most):
    for n in (most + 1, most + 15, most + 1000):
        assert status(name, defaults, spread(defaults, **sized(n))) == 1, n


@pytest.mark.parametrize("name,defaults,sized,most", LIMITS)
@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only where there is no device")
def test_counts_at_the_limit_get_as_far_as_the_device(name, defaults, sized, most):
    assert status(name, defaults, spread(defaults, **sized(most))) not in (0, 1, 2, 3)
