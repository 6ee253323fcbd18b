"""What the entry points of the sublayer in 8 bits take and refuse beside test_scaled_cpu's calls, without a GPU."""

import pytest
import torch

import newton_schulz_07_amd as ns
from tests.test_scaled_cpu import GRAD
from tests.test_sublayer_cpu import status

LINEAR = dict(experts=1, offsets=0)  # one expert that has all rows


@pytest.mark.parametrize("changes", [{}, dict(rows=0, n_x=30), dict(n_rows=0, rows=0, x=0, x_scales=0, dy=0)])
@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only where there is no device")
def test_a_linear_layers_weight_gradient_gets_as_far_as_the_device(changes):
    assert status("ns_experts_weight_grad_scaled", GRAD, {**LINEAR, **changes}) not in (0, 1, 2, 3), \
        ns.lib().ns_last_error().decode()


@pytest.mark.parametrize("changes,want", [(dict(experts=2), 1), (dict(rows=0), 1), (dict(dw=0), 1), (dict(offsets=2), 3)])
def test_a_linear_layers_weight_gradient_refuses(changes, want):
    assert status("ns_experts_weight_grad_scaled", GRAD, {**LINEAR, **changes}) == want
