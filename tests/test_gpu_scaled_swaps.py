"""GPU tests of the block-scaled product's FP8B rows from narrow tiles, whose largest
magnitudes the two CTAs of a pair swap: several tiles a pair, of all widths in
turn (a tile of up to 32 rows is one set's of warps alone), one or more slots of
scales a tile, wide tiles among them.  Definitions are test_gpu_scaled.py's."""
import numpy as np
import pytest
import torch

from test_gpu_scaled import check_product, make_rows, make_weights

pytestmark = pytest.mark.gpu

WIDTHS = (20, 33, 128, 1, 64, 65, 97, 32, 0, 100)  # rows of an expert, over and over


@pytest.fixture(scope="module")
def L():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return llmoe


def widths(E, T):
    c = np.array([[WIDTHS[(e * 7 + e // 10) % len(WIDTHS)]] for e in range(E)], np.int64)
    c[::11] = T  # where T is above 128: wide tiles
    return c


@pytest.mark.parametrize("T", [128, 300])
@pytest.mark.parametrize("n_in", [112, 528])
def test_every_width_in_turn(L, n_in, T):
    check_product(L, 1, T, 40, n_in, 1040, "fp8b", True, widths(40, T))


@pytest.mark.parametrize("T", [128, 300])
@pytest.mark.parametrize("n_in", [128, 640])
def test_the_same_bits_every_time(L, n_in, T):
    """Many tiles a pair, the caches cold and warm."""
    E, n_out = 96, 2048
    c = torch.from_numpy(widths(E, T)).cuda()
    x = make_rows(T * E // 32, n_in, 3)[0].repeat(32, 1)
    w, ws, _ = make_weights(4, 2, n_out, n_in, 4, 0.05)
    w, ws = w.repeat(E // 4, 1, 1, 1), ws.repeat(E // 4, 1, 1, 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bs = L.geometry(T, 1, E, err=err)
    flush = torch.empty(64 << 20, dtype=torch.float32, device="cuda")
    first = None
    for call in range(40):
        y = torch.zeros(E * T, L.llmoe_row_bytes(n_out, L.LLMOE_DTYPE_FP8B), dtype=torch.uint8, device="cuda")
        if call % 4 == 1:
            flush.add_(1)
        L.llmoe_expert_product_fp8b(x, w, ws, y, c, n_in, n_out, L.LLMOE_DTYPE_FP8B, L.LLMOE_PRODUCT_SWIGLU, bs)
        first = y if first is None else first
        assert torch.equal(first, y)
    assert int(err) == 0 and int(first.any(1).sum()) == int(c.sum())
