"""The router at every number of values a lane can hold: one expert above, at
and below each multiple of 128, against the FP64 form and bounds of
test_gpu_i8.py."""
import pytest
import torch
from test_gpu_i8 import check_route, cq, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", sorted({e for n in range(128, 1025, 128) for e in (n - 1, n, n + 1)}
                                     - {1025}) + [132, 388, 516, 644, 772, 900])
def test_route_at_the_borders_of_its_sizes(cq, E):  # noqa: F811
    g = gen(E)
    logits = torch.randn(9, E, generator=g, device="cuda") * 1.5
    logits[3] = 0.5                              # all equal
    logits[4, :E - 3] = float("-inf")            # the last ones only
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    for dt in (torch.float32, torch.bfloat16):
        for sigmoid in (False, True):
            for b in (None, bias):
                check_route(cq, logits.to(dt), 16, b, sigmoid, True)
