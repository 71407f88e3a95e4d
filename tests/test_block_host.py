"""Refusals of the block operators (include/llmoe_block.h): every call below
returns before anything is launched, so it runs without a GPU."""
import ctypes

import pytest

A = 1 << 24  # an aligned address; nothing dereferences it


@pytest.fixture(scope="module")
def lib():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    return llmoe


def test_row_bytes(lib):
    rb = lib.llmoe_row_bytes
    assert rb(7168, lib.LLMOE_DTYPE_BF16) == 14336 and rb(7168, lib.LLMOE_DTYPE_FP32) == 28672
    assert rb(7168, lib.LLMOE_DTYPE_MX8) == 7168 + 224
    assert rb(32, lib.LLMOE_DTYPE_MX8) == 48 and rb(512, lib.LLMOE_DTYPE_MX8) == 528 and rb(544, lib.LLMOE_DTYPE_MX8) == 576
    for n, t in [(0, 0), (-8, 0), (12, 0), (12, 1), (6, 2), (48, 3), (16, 3), (8, 4), (8, -1)]:
        assert rb(n, t) == 0, (n, t)


def norm(lib, **kw):
    a = dict(x=A, residual=2 * A, weight=3 * A, eps=1e-6, residual_out=2 * A, out=4 * A, rows=4, hidden=256, dtype=0,
             out_dtype=0)
    a.update(kw)
    return lib._lib.llmoe_add_rmsnorm(a["x"], a["residual"], a["weight"], a["eps"], a["residual_out"], a["out"],
                                      a["rows"], a["hidden"], a["dtype"], a["out_dtype"], None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(out=None), dict(weight=None), dict(x=A + 8), dict(residual=2 * A + 4), dict(out=4 * A + 2),
    dict(residual_out=2 * A + 2), dict(weight=3 * A + 1), dict(rows=-1), dict(hidden=0), dict(hidden=12), dict(hidden=-8),
    dict(hidden=32776), dict(dtype=3), dict(dtype=4), dict(out_dtype=1), dict(out_dtype=4), dict(eps=-1.0),
    dict(eps=float("nan")), dict(hidden=40, out_dtype=3), dict(rows=2**62),
    dict(out=A + 64), dict(out=2 * A), dict(out=3 * A), dict(out=A, out_dtype=3),  # out over x (shifted), residual, weight
    dict(residual_out=A + 16), dict(residual_out=4 * A), dict(residual_out=2 * A + 512), dict(residual_out=3 * A),
])
def test_norm_refusals(lib, kw):
    assert norm(lib, **kw) == lib.LLMOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("args", [
    (None, 2 * A, 4, 256, 0), (A, None, 4, 256, 0), (A + 2, 2 * A, 4, 256, 0), (A, 2 * A + 8, 4, 256, 0),
    (A, 2 * A, -1, 256, 0), (A, 2 * A, 4, 40, 0), (A, 2 * A, 4, 256, 3), (A, A, 4, 256, 0), (A, A + 1024, 4, 256, 0),
    (A, 2 * A, 4, 32800, 0),
])
def test_pack_refusals(lib, args):
    assert lib._lib.llmoe_pack_mx8(*args, None) == lib.LLMOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(topk_idx=None), dict(topk_w=None), dict(logits=A + 2), dict(bias=A + 1),
    dict(topk_idx=A + 4), dict(topk_w=A + 2), dict(rows=-1), dict(E=0), dict(E=8193), dict(K=0), dict(K=33, E=64),
    dict(K=9, E=8), dict(dtype=3), dict(dtype=-1), dict(scoring=2), dict(flags=2), dict(rows=2**62),
])
def test_router_refusals(lib, kw):
    a = dict(logits=A, bias=2 * A, active=3 * A, topk_idx=4 * A, topk_w=5 * A, rows=4, E=8, K=2, dtype=2, scoring=0,
             flags=1, scale=1.0)
    a.update(kw)
    assert lib._lib.llmoe_topk_router(*a.values(), None) == lib.LLMOE_ERR_INVALID_ARGUMENT


def product(lib, bs=None, **kw):
    a = dict(x=A, w=2 * A, y=3 * A, counts=4 * A, n_in=256, n_out=256, dtype=0, out_dtype=0, flags=0)
    a.update(kw)
    g = dict(num_max_tokens=8, num_ranks=2, num_experts=8)
    g.update(bs or {})
    s = lib.llmoe_buf_set_t(**g)
    return lib._lib.llmoe_expert_product(*a.values(), ctypes.byref(s), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(y=None), dict(x=A + 8), dict(w=2 * A + 8), dict(y=3 * A + 4), dict(counts=4 * A + 4),
    dict(n_in=0), dict(n_in=12), dict(n_out=0), dict(n_out=12), dict(n_in=-8), dict(n_out=-8), dict(dtype=2),
    dict(dtype=4), dict(out_dtype=1), dict(out_dtype=3), dict(dtype=1, out_dtype=0), dict(flags=2), dict(flags=4),
    dict(dtype=3, n_in=40), dict(dtype=3, out_dtype=3), dict(dtype=3, out_dtype=3, flags=1, n_out=40),
    dict(dtype=3, out_dtype=4), dict(out_dtype=-1), dict(flags=1, out_dtype=2, n_out=20),
    dict(y=A), dict(y=A + 512), dict(y=2 * A), dict(y=2 * A + 4096), dict(n_out=2**30 + 8),
    dict(counts=None),  # and no rank buffers to read them from
])
def test_product_refusals(lib, kw):
    assert product(lib, **kw) == lib.LLMOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bs", [
    dict(num_max_tokens=0), dict(num_ranks=0), dict(num_experts=0), dict(num_experts=9), dict(num_experts=1),
    dict(num_experts=8194), dict(err=A + 2), dict(num_max_tokens=2**28), dict(num_experts=8192, num_ranks=8192,
                                                                           num_max_tokens=64),
])
def test_product_geometry_refusals(lib, bs):
    assert product(lib, bs=bs) == lib.LLMOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bs", [
    dict(), dict(base=None), dict(base=A + 8), dict(rank_stride=1 << 12), dict(rank_stride=(1 << 20) + 8), dict(set=2),
    dict(set=-1), dict(hidden=0), dict(dtype=7),
])
def test_product_count_words_refusals(lib, bs):
    """counts NULL: the buffer set has to be one whose words can be read."""
    g = dict(base=A, rank_stride=1 << 20, hidden=256, dtype=0, set=0)
    if not bs:
        g = {}
    g.update(bs)
    assert product(lib, counts=None, bs=g) == lib.LLMOE_ERR_INVALID_ARGUMENT


def test_null_buffer_set(lib):
    assert lib._lib.llmoe_expert_product(A, 2 * A, 3 * A, 4 * A, 64, 64, 0, 0, 0, None, None) == \
        lib.LLMOE_ERR_INVALID_ARGUMENT
