"""Refusals of the block-scaled operators and of the router with groups: every
call returns before anything is launched, so it runs without a GPU."""
import ctypes

import pytest
import torch

A = 1 << 24  # an aligned address; nothing dereferences it


@pytest.fixture(scope="module")
def lib():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    return llmoe


def test_row_bytes(lib):
    rb, t = lib.llmoe_row_bytes, lib.LLMOE_DTYPE_FP8B
    assert rb(7168, t) == 7168 + 56 * 4 and rb(16, t) == 32 and rb(128, t) == 144 and rb(512, t) == 528
    assert rb(528, t) == 528 + 32 and rb(640, t) == 640 + 32  # five scales: 20 bytes
    for n in (0, -16, 8, 24, 130):
        assert rb(n, t) == 0, n


@pytest.mark.parametrize("args", [
    (None, 2 * A, 4, 256, 0), (A, None, 4, 256, 0), (A + 2, 2 * A, 4, 256, 0), (A, 2 * A + 8, 4, 256, 0),
    (A, 2 * A, -1, 256, 0), (A, 2 * A, 4, 40, 0), (A, 2 * A, 4, 256, 3), (A, 2 * A, 4, 256, 5), (A, A, 4, 256, 0),
    (A, A + 1024, 4, 256, 0), (A, 2 * A, 4, 32784, 0),
])
def test_pack_refusals(lib, args):
    assert lib._lib.llmoe_pack_fp8b(*args, None) == lib.LLMOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(out=None), dict(out=4 * A + 8), dict(hidden=264), dict(dtype=5), dict(out=A), dict(out=2 * A), dict(out=3 * A),
    dict(residual_out=4 * A + 1024), dict(hidden=32784),
])
def test_norm_refusals(lib, kw):
    a = dict(x=A, residual=2 * A, weight=3 * A, eps=1e-6, residual_out=2 * A, out=4 * A, rows=4, hidden=256, dtype=0,
             out_dtype=5)
    a.update(kw)
    assert lib._lib.llmoe_add_rmsnorm(*a.values(), None) == lib.LLMOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(w=None), dict(codes=None), dict(scales=None), dict(w=A + 8), dict(codes=2 * A + 8), dict(scales=3 * A + 2),
    dict(matrices=-1), dict(rows=0), dict(cols=0), dict(cols=24), dict(cols=-16), dict(dtype=3), dict(dtype=5),
    dict(matrices=2**60), dict(codes=A), dict(codes=A + 256), dict(scales=A), dict(scales=2 * A + 64),
])
def test_pack_weights_refusals(lib, kw):
    a = dict(w=A, codes=2 * A, scales=3 * A, matrices=2, rows=40, cols=48, dtype=0)
    a.update(kw)
    assert lib._lib.llmoe_pack_fp8b_weights(*a.values(), None) == lib.LLMOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(topk_idx=None), dict(topk_w=None), dict(logits=A + 2), dict(bias=A + 1),
    dict(topk_idx=4 * A + 4), dict(topk_w=5 * A + 2), dict(rows=-1), dict(E=0), dict(E=8200), dict(K=0), dict(K=33, E=64),
    dict(K=9), dict(dtype=3), dict(dtype=-1), dict(scoring=2), dict(flags=4), dict(rows=2**62),
    dict(groups=0), dict(groups=3), dict(groups=32), dict(groups=512, E=1024), dict(kept=0), dict(kept=5),
    dict(kept=1, K=5), dict(scoring=1, flags=2), dict(topk_idx=A), dict(topk_w=4 * A + 8), dict(topk_w=2 * A),
    dict(topk_idx=3 * A),
])
def test_router_refusals(lib, kw):
    a = dict(logits=A, bias=2 * A, active=3 * A, topk_idx=4 * A, topk_w=5 * A, rows=4, E=16, K=2, groups=4, kept=2,
             dtype=2, scoring=0, flags=3, scale=1.0)
    a.update(kw)
    assert lib._lib.llmoe_group_router(*a.values(), None) == lib.LLMOE_ERR_INVALID_ARGUMENT


def product(lib, bs=None, **kw):
    a = dict(x=A, w=2 * A, scale=5 * A, y=3 * A, counts=4 * A, n_in=256, n_out=256, out_dtype=0, flags=0)
    a.update(kw)
    g = dict(num_max_tokens=8, num_ranks=2, num_experts=8)
    g.update(bs or {})
    s = lib.llmoe_buf_set_t(**g)
    return lib._lib.llmoe_expert_product_fp8b(*a.values(), ctypes.byref(s), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(scale=None), dict(y=None), dict(x=A + 8), dict(w=2 * A + 8), dict(scale=5 * A + 2),
    dict(y=3 * A + 4), dict(counts=4 * A + 4), dict(n_in=0), dict(n_in=24), dict(n_out=0), dict(n_out=12), dict(n_in=-16),
    dict(n_out=-8), dict(out_dtype=3), dict(out_dtype=4), dict(out_dtype=5), dict(out_dtype=-1), dict(flags=2),
    dict(out_dtype=5, flags=1, n_out=40), dict(flags=1, out_dtype=2, n_out=20), dict(y=A), dict(y=A + 512),
    dict(y=2 * A), dict(y=2 * A + 4096), dict(y=5 * A), dict(n_out=2**30 + 8), dict(n_in=2**31 - 16, n_out=2**29),
    dict(counts=None),  # and no rank buffers to read them from
])
def test_product_refusals(lib, kw):
    assert product(lib, **kw) == lib.LLMOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bs", [
    dict(num_max_tokens=0), dict(num_ranks=0), dict(num_experts=0), dict(num_experts=9), dict(num_experts=1),
    dict(num_experts=8194), dict(err=A + 2), dict(num_max_tokens=2**28),
])
def test_product_geometry_refusals(lib, bs):
    assert product(lib, bs=bs) == lib.LLMOE_ERR_INVALID_ARGUMENT


def test_other_products_refuse_the_row_type(lib):
    g = lib.llmoe_buf_set_t(num_max_tokens=8, num_ranks=2, num_experts=8)
    for dtype, out, flags in [(5, 0, 0), (5, 5, 1), (0, 5, 1), (3, 5, 1), (3, 5, 0), (1, 5, 0)]:
        assert lib._lib.llmoe_expert_product(A, 2 * A, 3 * A, 4 * A, 256, 256, dtype, out, flags, ctypes.byref(g),
                                             None) == lib.LLMOE_ERR_INVALID_ARGUMENT
    assert lib._lib.llmoe_pack_mx8(A, 2 * A, 4, 256, 5, None) == lib.LLMOE_ERR_INVALID_ARGUMENT
    assert lib.llmoe_layout_bytes_dtype(8, 64, 1, 8, 5) == 0  # no payload type


def test_python_argument_types(lib):
    codes = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        lib.llmoe_pack_fp8b_weights(torch.zeros(1, 16), codes, torch.zeros(1), 1, 1, 16, lib.LLMOE_DTYPE_FP32, 0)
    with pytest.raises(ValueError):
        lib.llmoe_group_router(torch.zeros(1, 16), None, None, codes, codes, 1, 16, 1, 2, 1, lib.LLMOE_DTYPE_FP32, 0, 0,
                               1.0, 0)


T, R, H, I, E, K = 6, 2, 64, 48, 8, 2
z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
f32, u8 = torch.float32, torch.uint8
CODED = dict(gate_up=z(E, 2 * I, H, dtype=u8), down=z(E, H, I, dtype=u8), gate_up_scale=z(E, 2, 1, 1, dtype=f32),
             down_scale=z(E, 1, 1, dtype=f32), rows="fp8b")


@pytest.mark.parametrize("what,kw", [
    ("num_groups", dict(num_groups=0)), ("num_groups", dict(num_groups=3)),
    ("kept_groups", dict(num_groups=4, kept_groups=5)), ("kept_groups", dict(num_groups=4, kept_groups=0)),
    ("kept_groups", dict(num_groups=8, kept_groups=1)),
    ("group_top2", dict(num_groups=4, kept_groups=2, group_top2=True, scoring=1)),
    ("hidden", dict(rows="fp8b", gate_up=z(E, 2 * 40, H), down=z(E, H, 40))),
    ("gate_up_scale", dict(CODED, gate_up_scale=None)), ("down_scale", dict(CODED, down_scale=None)),
    ("gate_up_scale", dict(CODED, rows="mx8")), ("gate_up_scale", dict(CODED, rows="same")),
    ("gate_up_scale", dict(CODED, gate_up_scale=z(E, 1, 1, dtype=f32))),
    ("gate_up_scale", dict(CODED, gate_up_scale=z(E, 2, 1, 1))),
    ("down_scale", dict(CODED, down_scale=z(E, 1, 2, dtype=f32))),
    ("gate_up", dict(CODED, gate_up=z(E, 2 * I, H))), ("down", dict(CODED, down=z(E, I, H, dtype=u8).transpose(1, 2))),
])
def test_block_refusals(lib, what, kw):
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    a = dict(num_max_tokens=T, num_ranks=R, num_topk=K, norm_weight=z(H), router_weight=z(E, H), gate_up=z(E, 2 * I, H),
             down=z(E, H, I))
    a.update(kw)
    with pytest.raises(ValueError, match=rf"\b{what}\b"):
        MoEBlock(**a)


@pytest.mark.parametrize("what,w", [("16 bytes", z(2, 4, 24)), ("bf16", z(2, 4, 32, dtype=torch.float64)),
                                    ("no matrices", z(32)), ("no matrices", z(2, 0, 32)), ("no matrices", z(2, 4, 0)),
                                    ("CUDA", z(2, 4, 32))])
def test_weight_packing_refusals(lib, what, w):
    from combine_routing_count_prefix_gb300.moe_block import pack_fp8b_weights

    with pytest.raises(ValueError, match=what):
        pack_fp8b_weights(w)
