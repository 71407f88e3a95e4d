"""Refusals of llmoe_topk_router where its outputs overlap its inputs or each
other: it returns before anything is launched, so this runs without a GPU."""
import pytest

A = 1 << 24  # an aligned address; nothing dereferences it
ROWS, E, K = 4, 8, 2
LOGITS, BIAS, ACTIVE, IDX, W = A, 2 * A, 3 * A, 4 * A, 5 * A


@pytest.fixture(scope="module")
def lib():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    return llmoe


@pytest.mark.parametrize("dtype", [0, 2])
@pytest.mark.parametrize("kw", [
    dict(topk_idx=LOGITS), dict(topk_w=LOGITS), dict(topk_idx=LOGITS - ROWS * K * 8 + 8), dict(topk_w=LOGITS + ROWS * E * 2 - 4),
    dict(topk_idx=BIAS), dict(topk_w=BIAS + E * 4 - 4), dict(topk_idx=ACTIVE), dict(topk_w=ACTIVE - ROWS * K * 4 + 4),
    dict(topk_w=IDX), dict(topk_w=IDX + ROWS * K * 8 - 4), dict(topk_idx=W - 8),
    dict(bias=IDX + 16), dict(active=W + 1),
])
def test_overlap(lib, kw, dtype):
    a = dict(logits=LOGITS, bias=BIAS, active=ACTIVE, topk_idx=IDX, topk_w=W)
    a.update(kw)
    assert lib._lib.llmoe_topk_router(*a.values(), ROWS, E, K, dtype, 0, 1, 1.0, None) == lib.LLMOE_ERR_INVALID_ARGUMENT
