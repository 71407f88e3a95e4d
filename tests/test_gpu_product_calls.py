"""GPU test of what a product call costs on the host: nothing is asked of the
driver again because the previous call had another shape.

Asking again (occupancy, shared-memory opt-in) takes 0.6 us, 12% of a call of
5.3 us; a call is timed by itself and in turn with one of another number of
experts, in pairs of measurements, and the median of 60 ratios may be 1.06, half
of that.
"""
import statistics
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return llmoe


def test_calls_of_two_shapes_in_turn(L):
    keep = []

    def call(E):
        x, w, y = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((E * 8, 64), (E, 64, 64), (E * 8, 64)))
        counts = torch.ones(E, 1, dtype=torch.int64, device="cuda")
        bs = L.geometry(8, 1, E)
        keep.append((x, w, y, counts, bs))
        return lambda: L.llmoe_expert_product(x, w, y, counts, 64, 64, 0, 0, 0, bs)

    a, b = call(1), call(8)

    def host_time(first, second):
        torch.cuda.synchronize()
        begin = time.perf_counter()
        for _ in range(100):  # far fewer than a stream's queue holds
            first()
            second()
        return time.perf_counter() - begin

    for pair in ((a, a), (b, b), (a, b)):
        host_time(*pair)
    ratios = []
    for _ in range(60):
        alone = host_time(a, a) + host_time(b, b)
        ratios.append(2 * host_time(a, b) / alone)
    assert statistics.median(ratios) <= 1.06, statistics.quantiles(ratios)
