"""GPU tests of the block-scaled product's wide tiles (more than 128 padded rows of
an expert: the rows on the tensor core's M side), whose sums, scales and stores
are their own: every output type, outputs whose last 32 bytes are half full, and
NaN and infinite scales.  Definitions and tolerances are test_gpu_scaled.py's."""
import numpy as np
import pytest
import torch

import fp8b_reference as fp8b
import test_gpu_scaled
from test_gpu_scaled import check_product, make_rows, make_weights

pytestmark = pytest.mark.gpu

GROUP, NARROW = 4, 128  # rows taken together; rows of the largest narrow tile


@pytest.fixture(scope="module")
def L():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return llmoe


def close(got, want, err, dtype, close=test_gpu_scaled.close):
    """The same, with fp16's infinities: its largest is 65504 and its steps there are 32,
    so a value of 65520 or more rounds to infinity and one below to 65504 at most.
    (A row's values are of a size of their own; SwiGLU's are squares of it.)"""
    if dtype == "fp16":
        over = np.isinf(got)
        assert ((np.sign(got) * want + err)[over] >= 65520).all()
        assert not (np.abs(want) - err >= 65520)[~over].any()
        got, want, err = got[~over], want[~over], err[~over]
    close(got, want, err, dtype)


@pytest.fixture(autouse=True)
def _with_infinities(monkeypatch):
    monkeypatch.setattr(test_gpu_scaled, "close", close)


def groups(counts):
    return (-(-counts // GROUP)).sum(1)


# in: one step, two, five, nine (of 128); out by type: one block and less, the last 32
# bytes half full, past a block and past a tile
SIZES = {"bf16": (8, 264), "fp16": (40, 520), "fp32": (4, 132), "fp8b": (16, 176)}


@pytest.mark.parametrize("out_dtype,swiglu", [("bf16", False), ("fp16", False), ("fp32", False), ("bf16", True),
                                              ("fp16", True), ("fp32", True), ("fp8b", True)])
@pytest.mark.parametrize("n_in", [16, 144, 640, 1040])
@pytest.mark.parametrize("R,T", [(1, 300), (2, 140)])
def test_types_and_sizes(L, R, T, n_in, out_dtype, swiglu):
    for n_out in SIZES[out_dtype]:
        if swiglu and n_out % 8:
            n_out += 4  # whole eights of gate and up
        counts = np.full((2, R), T, np.int64)
        counts[1] = np.random.RandomState(n_in).randint(T // 2 + 24, T, R)  # ends inside a warp's rows
        assert (groups(counts) * GROUP > NARROW).all()
        check_product(L, R, T, 2, n_in, n_out, out_dtype, swiglu, counts)


@pytest.mark.parametrize("out_dtype,swiglu", [("bf16", False), ("fp32", False), ("bf16", True), ("fp32", True),
                                              ("fp8b", True)])
def test_kinds_of_tiles_in_turn(L, out_dtype, swiglu):
    """Wide tiles, tiles of every narrow width and experts without rows, several of
    them a pair: buffers change their size and the kinds' own barriers stay in step."""
    R, T, E = 2, 150, 12
    counts = np.array([[150, 150], [1, 0], [70, 62], [0, 0], [140, 3], [30, 30], [128, 0], [129, 0], [0, 33], [64, 64],
                       [97, 150], [2, 3]], np.int64)
    check_product(L, R, T, E, 400, 2064, out_dtype, swiglu, counts)


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32", "fp8b"])
def test_nan_stays_in_its_row_and_block(L, out_dtype):
    R, T, E, n_in, n_out = 1, 200, 2, 256, 256
    counts = np.array([[200], [150]], np.int64)
    assert (groups(counts) > NARROW // GROUP).all()
    swiglu = out_dtype == "fp8b"
    x, _ = make_rows(E * R * T, n_in, 1)
    w, ws, _ = make_weights(E, 1 + swiglu, n_out, n_in, 2, 0.1)
    code = L.ROW_DTYPE_CODES[out_dtype]
    c = torch.from_numpy(counts).cuda()

    def run():
        y = torch.zeros(E * R * T, L.llmoe_row_bytes(n_out, code), dtype=torch.uint8, device="cuda")
        L.llmoe_expert_product_fp8b(x, w, ws, y, c, n_in, n_out, code, int(swiglu), L.geometry(T, R, E))
        return y.cpu()

    clean = run()
    bad = [5, 6, 70, 199]
    x[5, n_in:n_in + 4] = 255  # a NaN scale of the first block of 128 values
    x[6, 3] = 127  # a NaN code
    x[70, n_in + 4:n_in + 8] = 255  # a NaN scale of the second
    x[199, 255] = 255  # a NaN code in the last row, last value
    ws[1, 0, 1, 0] = float("inf")  # features 128.. of expert 1 (with SwiGLU its gate)
    got = run()
    same = np.ones(E * T, bool)
    same[bad] = False
    same[T:] = False
    assert torch.equal(got[torch.from_numpy(same)], clean[torch.from_numpy(same)])
    hit = slice(T, T + 150)
    assert not got[T + 150:].any()
    if swiglu:
        q, s, _ = fp8b.split(got.numpy(), n_out)
        assert np.isnan(s[bad]).all() and np.isnan(q[bad]).all()
        assert np.isnan(s[hit, 1]).all()
        assert torch.equal(got[hit, :128], clean[hit, :128])
        assert torch.equal(got[hit, n_out:n_out + 4], clean[hit, n_out:n_out + 4])
    else:
        t = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        v, k = got.view(t), clean.view(t)
        assert v[bad].isnan().all()
        assert torch.equal(v[hit, :128], k[hit, :128]) and not v[hit, 128:].isfinite().any()
