"""GPU tests of the block operators (norm, router, expert products) against
their definitions in 64 bits (tests/block_reference.py).

Tolerances, derived from the arithmetic each call documents:
- fp32 norm: a thread sums at most 64 squares in a row, then ten levels of
  pairwise sums; halved by the square root, plus a square root, a division and
  two products: 48 roundings of 2^-24, 3e-6 in all;
- a result rounded to bf16 / fp16 / fp32 may be off by half an ulp more
  (of 8, 11 and 24 significant bits: 2^-8, 2^-11 and 2^-24 of the value; the
  least subnormal's half below);
- router weights: exponential, sum and division, one rounding each per term;
- products: an fp32 sum of n products, each addition within 2^-23 of the sum
  of the magnitudes (the tensor cores truncate), and the rounding to the output
  type.
"""
import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_ULP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}
NORM_ERR = 3e-6


@pytest.fixture(scope="module")
def L():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return llmoe


def rnd(seed):
    return torch.Generator().manual_seed(seed)


def wide(t):
    return t.cpu().to(torch.float64).numpy()


def close(got, want, err, dtype):
    """got within err of want, and half an ulp of dtype (of got's size)."""
    tol = err + (np.abs(want) + err) * HALF_ULP[dtype] + TINY[dtype]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.abs(got - want)[bad][:4], tol[bad][:4])


# ---------------------------------------------------------------------------
# rows: norm and packing
# ---------------------------------------------------------------------------

NORM_SHAPES = [(1, 64), (3, 96), (5, 2048), (2, 7168), (1, 32768), (700, 224), (2048, 32), (410, 7168), (1300, 2080),
               (153, 16384), (160, 32768)]


@pytest.mark.parametrize("out", ["same", "mx8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,hidden", NORM_SHAPES)
def test_add_rmsnorm(L, rows, hidden, dtype, out):
    g = rnd(rows * 7 + hidden)
    x = torch.randn(rows, hidden, generator=g).to(TORCH[dtype])
    res = (3 * torch.randn(rows, hidden, generator=g)).to(TORCH[dtype])
    w = (1 + 0.2 * torch.randn(hidden, generator=g)).to(TORCH[dtype])
    x[rows // 2] = 0  # a row whose sum may be the residual alone
    if rows > 1:
        res[0] = -x[0]  # and one whose sum is zero: eps alone under the root
    h = (x.float() + res.float()).to(TORCH[dtype])
    od = dtype if out == "same" else "mx8"
    code = L.ROW_DTYPE_CODES
    rb = L.llmoe_row_bytes(hidden, code[od])
    got = torch.full((rows * rb + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    hout = torch.empty_like(x, device="cuda")
    L.llmoe_add_rmsnorm(x.cuda(), res.cuda(), w.cuda(), 1e-5, hout, got[:-16], rows, hidden, code[dtype], code[od])
    assert torch.equal(hout.cpu(), h)
    assert (got[-16:] == 0xA5).all()
    v = ref.rmsnorm(wide(h), wide(w), 1e-5)
    if out == "mx8":
        ref.check_mx8(got[:-16].reshape(rows, rb).cpu().numpy(), v, np.abs(v) * NORM_ERR)
    else:
        close(wide(got[:-16].view(TORCH[dtype]).reshape(rows, hidden)), v, np.abs(v) * NORM_ERR, dtype)


@pytest.mark.parametrize("rows,hidden", [(37, 1056), (900, 1056), (350, 4104)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_add_rmsnorm_in_place_and_without_residual(L, dtype, rows, hidden):
    g = rnd(5)
    x = torch.randn(rows, hidden, generator=g).to(TORCH[dtype])
    res = torch.randn(rows, hidden, generator=g).to(TORCH[dtype])
    w = torch.randn(hidden, generator=g).to(TORCH[dtype])
    c = L.ROW_DTYPE_CODES[dtype]
    # no residual: h = x; out over x
    a = x.cuda()
    L.llmoe_add_rmsnorm(a, None, w.cuda(), 0.0, None, a, rows, hidden, c, c)
    v = ref.rmsnorm(wide(x), wide(w), 0.0)
    close(wide(a), v, np.abs(v) * NORM_ERR, dtype)
    # the stored sum over the residual, then over x
    h = (x.float() + res.float()).to(TORCH[dtype])
    v = ref.rmsnorm(wide(h), wide(w), 1e-6)
    for over in ("residual", "x"):
        a, b, o = x.cuda(), res.cuda(), torch.empty_like(x, device="cuda")
        L.llmoe_add_rmsnorm(a, b, w.cuda(), 1e-6, b if over == "residual" else a, o, rows, hidden, c, c)
        assert torch.equal((b if over == "residual" else a).cpu(), h)
        close(wide(o), v, np.abs(v) * NORM_ERR, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,hidden", [(1, 32), (9, 512), (4, 7168), (3, 544), (500, 1056), (5000, 96)])
def test_pack_mx8_is_exact(L, rows, hidden, dtype):
    g = rnd(rows + hidden)
    x = (torch.randn(rows, hidden, generator=g) * torch.exp2(torch.randint(-12, 9, (rows, hidden // 32, 1), generator=g)
         .float()).expand(-1, -1, 32).reshape(rows, hidden)).to(TORCH[dtype])
    x[0, :32] = 0  # a group of zeros
    if hidden >= 512:
        x[0, 32:64] = 0
        x[0, 32] = 448  # exactly e4m3's largest at scale 1
        x[0, 64:96] = 0
        x[0, 64] = -452  # above it: the next scale
        x[0, 96:128] = torch.tensor([17.0, 19.0, 21.0, 23.0] * 8) / 16  # midpoints of e4m3 at some scales
        x[0, 96] = 448
    got = torch.empty(rows, L.llmoe_row_bytes(hidden, L.LLMOE_DTYPE_MX8), dtype=torch.uint8, device="cuda")
    L.llmoe_pack_mx8(x.cuda(), got, rows, hidden, L.ROW_DTYPE_CODES[dtype])
    want = ref.pack_mx8(wide(x))
    got = got.cpu().numpy()
    assert np.array_equal(got[:, hidden:], want[:, hidden:])
    assert np.array_equal(ref.E4M3[got[:, :hidden]], ref.E4M3[want[:, :hidden]])


def test_pack_mx8_of_nan_and_infinity(L):
    x = torch.ones(1, 128, dtype=torch.bfloat16)
    x[0, 5], x[0, 70] = float("nan"), float("-inf")
    got = torch.empty(1, 144, dtype=torch.uint8, device="cuda")
    L.llmoe_pack_mx8(x.cuda(), got, 1, 128, L.LLMOE_DTYPE_BF16)
    assert got.cpu()[0, 128:132].tolist() == [255, 119, 255, 119]  # 1 = 256 * 2^-8


def test_norm_no_rows(L):
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    L.llmoe_add_rmsnorm(None, None, w, 1e-6, None, None, 0, 64, 0, 0)
    L.llmoe_pack_mx8(None, None, 0, 64, 0)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------

def run_router(L, logits, bias, active, K, dtype, scoring, renorm, scale):
    rows, E = logits.shape
    idx = torch.full((rows, K), -7, dtype=torch.int64, device="cuda")
    w = torch.full((rows, K), float("nan"), device="cuda")
    L.llmoe_topk_router(logits.cuda(), None if bias is None else bias.cuda(), None if active is None else active.cuda(),
                        idx, w, rows, E, K, L.DTYPE_CODES[dtype],
                        L.LLMOE_SCORE_SIGMOID if scoring == "sigmoid" else L.LLMOE_SCORE_SOFTMAX,
                        L.LLMOE_ROUTER_RENORM if renorm else 0, scale)
    return idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("scoring,bias", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,E,K", [(1, 1, 1), (5, 8, 8), (3, 33, 2), (64, 64, 6), (17, 256, 8), (9, 511, 32),
                                      (4, 513, 8), (3, 2049, 9), (2, 8192, 32)])
def test_router(L, rows, E, K, dtype, scoring, bias):
    g = rnd(rows * 31 + E)
    # eighths: exact in every type, and so many that keys tie
    logits = torch.randint(-24, 25, (rows, E), generator=g).float() / 8
    b = torch.randint(-1, 2, (E,), generator=g).float() / 4 if bias else None
    active = (torch.rand(rows, generator=g) < 0.8).to(torch.uint8) if rows > 4 else None
    renorm = rows % 2 == 1
    idx, w, gap = ref.router(logits.numpy(), None if b is None else b.numpy(), None if active is None else active.numpy(),
                             K, scoring, renorm, 2.5)
    assert gap > 1e-6  # so that fp32 keys order as the exact ones do
    gi, gw = run_router(L, logits.to(TORCH[dtype]), b, active, K, dtype, scoring, renorm, 2.5)
    assert np.array_equal(gi, idx)
    assert (np.abs(gw - w) <= w * (E / 32 + K + 32) * 2.0 ** -23).all()


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,K,spread", [(256, 8, 1.0), (256, 8, 12.0), (128, 6, 3.0), (60, 8, 1.0), (512, 32, 1.0)])
def test_router_continuous_logits(L, E, K, spread, scoring):
    """Keys without a grid: rows whose K + 1 largest are 1e-6 apart choose as the exact ones do."""
    rows = 400
    g = rnd(E + K)
    logits = torch.randn(rows, E, generator=g) * spread
    b = torch.randn(E, generator=g) * 0.3
    gi, gw = run_router(L, logits, b, None, K, "fp32", scoring, True, 1.0)
    seen = 0
    for r in range(rows):
        idx, w, gap = ref.router(logits[r:r + 1].numpy(), b.numpy(), None, K, scoring, True, 1.0)
        key = 1 / (1 + np.exp(-logits[r].double().numpy())) if scoring == "sigmoid" else logits[r].double().numpy()
        near = np.sort(key + b.double().numpy())[::-1][:K + 1]
        if np.diff(-near).min() < 1e-5 * max(1.0, spread):
            continue
        seen += 1
        assert np.array_equal(gi[r], idx[0]), r
        assert (np.abs(gw[r] - w[0]) <= w[0] * (E / 32 + K + 32 + 2 * np.abs(logits[r].numpy()).max()) * 2.0 ** -23).all()
    assert seen > rows // 2


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_router_masked_experts(L, scoring):
    inf, nan = float("inf"), float("nan")
    E, K = 40, 4
    logits = torch.zeros(6, E)
    logits[0] = -inf  # nothing can be chosen
    logits[1] = -inf
    logits[1, 7], logits[1, 39] = 0.5, 1.5  # two can
    logits[2] = nan
    logits[2, 3] = -2.0
    logits[3, 20:] = nan  # NaN beside ordinary ones
    logits[4, 11] = logits[4, 30] = inf  # two of the largest
    logits[5] = torch.finfo(torch.float32).min  # a mask of the type's lowest value, over the whole row
    bias = torch.zeros(E)
    bias[2] = -inf  # masked by the bias
    for b in (None, bias):
        idx, w, _ = ref.router(np.where(np.isnan(logits.numpy()), -np.inf, logits.numpy()),
                               None if b is None else b.numpy(), None, K, scoring, True, 1.0)
        gi, gw = run_router(L, logits, b, None, K, "fp32", scoring, True, 1.0)
        assert np.array_equal(gi, idx)
        assert np.allclose(gw, w, rtol=64 * 2.0 ** -23, atol=0)


@pytest.mark.parametrize("E", [256, 100, 257])
def test_router_logits_not_16_byte_aligned(L, E):
    rows, K = 70, 8
    flat = torch.randint(-24, 25, (rows * E + 1,), generator=rnd(E)).float() / 8
    at = flat.cuda()[1:]
    idx = torch.empty(rows, K, dtype=torch.int64, device="cuda")
    w = torch.empty(rows, K, device="cuda")
    L.llmoe_topk_router(at, None, None, idx, w, rows, E, K, L.LLMOE_DTYPE_FP32, L.LLMOE_SCORE_SOFTMAX, 0, 1.0)
    want, ww, _ = ref.router(flat[1:].reshape(rows, E).numpy(), None, None, K, "softmax", False, 1.0)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert (np.abs(w.cpu().double().numpy() - ww) <= ww * (E / 32 + K + 32) * 2.0 ** -23).all()


def test_router_no_rows(L):
    L.llmoe_topk_router(None, None, None, None, None, 0, 8, 2, L.LLMOE_DTYPE_FP32, 0, 0, 1.0)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# expert products
# ---------------------------------------------------------------------------

def some_counts(E, R, T, kind, seed):
    r = np.random.RandomState(seed)
    if kind == "full":
        return np.full((E, R), T, np.int64)
    if kind == "none":
        return np.zeros((E, R), np.int64)
    if kind == "one":  # a single row in the whole call
        c = np.zeros((E, R), np.int64)
        c[E - 1, R // 2] = 1
        return c
    c = r.randint(0, T + 1, (E, R))
    c[r.rand(E, R) < 0.3] = 0
    c[r.randint(E)] = 0  # an expert without rows
    c[r.randint(E), r.randint(R)] = T
    return c.astype(np.int64)


def make_rows(L, n_rows, n, dtype, seed, scale=1.0):
    """Device rows of a row type and their 64-bit values."""
    v = torch.randn(n_rows, n, generator=rnd(seed)) * scale
    if dtype == "mx8":
        rows = ref.pack_mx8(v.double().numpy())
        return torch.from_numpy(rows).cuda(), ref.mx8_values(rows, n)
    t = v.to(TORCH[dtype])
    return t.cuda(), wide(t)


def check_product(L, R, T, E, n_in, n_out, dtype, out_dtype, swiglu, counts, bs=None, call_counts="given", stream=None):
    rows = E * R * T
    x, xv = make_rows(L, rows, n_in, dtype, 11 * E + n_in)
    w, wv = make_rows(L, E * n_out * (1 + swiglu), n_in, dtype, 13 * E + n_out, n_in ** -0.5)
    at, v, err = ref.product(xv, wv.reshape(E, -1, n_in), counts, T, swiglu)
    # rows that were not received hold anything: NaN here (0xFF codes and scales)
    unused = np.ones(rows, bool)
    unused[at] = False
    if dtype == "mx8":
        x[torch.from_numpy(unused)] = 0xFF
    else:
        x[torch.from_numpy(unused)] = float("nan")
    code = L.ROW_DTYPE_CODES
    rb = L.llmoe_row_bytes(n_out, code[out_dtype])
    y = torch.full((rows + 1, rb), 0xA5, dtype=torch.uint8, device="cuda")
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    if bs is None:
        bs = L.geometry(T, R, E, err=e)
    c = torch.from_numpy(counts).cuda() if call_counts == "given" else None
    torch.cuda.synchronize()
    L.llmoe_expert_product(x, w, y[:rows], c, n_in, n_out, code[dtype], code[out_dtype],
                           L.LLMOE_PRODUCT_SWIGLU if swiglu else 0, bs, stream)
    torch.cuda.synchronize()
    assert int(e) == 0
    y = y.cpu()
    assert (y[rows] == 0xA5).all() and (y[:rows][torch.from_numpy(unused)] == 0xA5).all()
    got = y[:rows][torch.from_numpy(at)]
    if not len(at):
        return
    if out_dtype == "mx8":
        ref.check_mx8(got.numpy(), v, err)
    else:
        close(wide(got.contiguous().view(TORCH[out_dtype])), v, err, out_dtype)


PRODUCT_TYPES = [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("mx8", "bf16"), ("mx8", "fp16"),
                 ("mx8", "fp32"), ("mx8", "mx8")]
# in, out: below one tile, odd multiples, one tile, past a tile's edge in either
PRODUCT_SIZES = [(32, 32), (96, 160), (128, 256), (544, 288), (256, 32)]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", PRODUCT_TYPES)
@pytest.mark.parametrize("n_in,n_out", PRODUCT_SIZES)
def test_product_types_and_sizes(L, n_in, n_out, dtype, out_dtype, swiglu):
    if out_dtype == "mx8" and not swiglu:
        pytest.skip("MX8 output belongs to the SwiGLU product")
    R, T, E = 2, 21, 4
    check_product(L, R, T, E, n_in, n_out, dtype, out_dtype, swiglu, some_counts(E, R, T, "ragged", n_in))


@pytest.mark.parametrize("kind", ["ragged", "full", "none", "one"])
@pytest.mark.parametrize("dtype", ["bf16", "mx8"])
@pytest.mark.parametrize("R,T,E", [(1, 1, 1), (1, 300, 3), (8, 5, 16), (40, 3, 40), (4, 130, 4), (3, 1, 96)])
def test_product_geometries(L, R, T, E, dtype, kind):
    out_dtype = "bf16"
    check_product(L, R, T, E, 160, 96, dtype, out_dtype, False, some_counts(E, R, T, kind, R + T))
    check_product(L, R, T, E, 160, 96, dtype, "mx8" if dtype == "mx8" else out_dtype, True,
                  some_counts(E, R, T, kind, R + T + 1))


@pytest.mark.parametrize("n_in,n_out,swiglu", [(8, 8, False), (24, 40, True), (72, 520, False), (1032, 264, True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_product_odd_sizes_16_bit(L, n_in, n_out, swiglu, dtype):
    check_product(L, 2, 33, 4, n_in, n_out, dtype, dtype, swiglu, some_counts(4, 2, 33, "ragged", 3))


@pytest.mark.parametrize("dtype", ["bf16", "mx8"])
def test_product_long_inner_dimension(L, dtype):
    check_product(L, 1, 40, 2, 4096, 64, dtype, "bf16", False, some_counts(2, 1, 40, "full", 0))


def test_product_on_another_stream(L):
    s = torch.cuda.Stream()
    check_product(L, 2, 17, 4, 128, 128, "bf16", "bf16", True, some_counts(4, 2, 17, "ragged", 9), stream=s)


@pytest.mark.parametrize("dtype", ["bf16", "mx8"])
def test_product_is_reproducible_and_captures(L, dtype):
    """The same bits on every call, eager and replayed from a CUDA graph."""
    R, T, E, n_in, n_out = 2, 70, 6, 256, 320
    x, _ = make_rows(L, E * R * T, n_in, dtype, 1)
    w, _ = make_rows(L, E * 2 * n_out, n_in, dtype, 2, 0.1)
    c = torch.from_numpy(some_counts(E, R, T, "ragged", 4)).cuda()
    code = L.ROW_DTYPE_CODES
    bs = L.geometry(T, R, E)
    ys = [torch.zeros(E * R * T, n_out, dtype=torch.bfloat16, device="cuda") for _ in range(3)]

    def call(y):
        L.llmoe_expert_product(x, w, y, c, n_in, n_out, code[dtype], code["bf16"], L.LLMOE_PRODUCT_SWIGLU, bs)

    call(ys[0])
    call(ys[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ys[2])
    ys[2].fill_(0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("mx8", "bf16"), ("mx8", "mx8")])
def test_product_nan_stays_in_its_row_and_feature(L, dtype, out_dtype):
    R, T, E, n_in, n_out = 1, 40, 2, 256, 128
    counts = torch.tensor([[40], [7]], dtype=torch.int64, device="cuda")
    swiglu = out_dtype == "mx8"
    x, _ = make_rows(L, E * R * T, n_in, dtype, 1)
    w, _ = make_rows(L, E * n_out * (1 + swiglu), n_in, dtype, 2, 0.1)
    code = L.ROW_DTYPE_CODES
    rb = L.llmoe_row_bytes(n_out, code[out_dtype])

    def run():
        y = torch.zeros(E * R * T, rb, dtype=torch.uint8, device="cuda")
        L.llmoe_expert_product(x, w, y, counts, n_in, n_out, code[dtype], code[out_dtype], int(swiglu), L.geometry(T, R, E))
        return y.cpu()

    clean = run()
    if dtype == "mx8":
        x[5, n_in + 3] = 255  # the NaN scale of one group
        w[n_out * (1 + swiglu) + 9, n_in] = 255  # feature (or gate) 9 of expert 1
    else:
        x[5, 100] = float("nan")
        w[n_out + 9, 0] = float("inf")
    got = run()
    same = np.ones(E * T, bool)
    same[5] = False
    same[T:T + 7] = False
    assert torch.equal(got[torch.from_numpy(same)], clean[torch.from_numpy(same)])
    if out_dtype == "mx8":
        assert (got[5, n_out:n_out + n_out // 32] == 255).all()  # every group holds a NaN
        hit = got[T:T + 7]
        assert (hit[:, n_out] == 255).all()  # the group of feature 9, and no other
        assert torch.equal(hit[:, 32:n_out], clean[T:T + 7, 32:n_out])
        assert torch.equal(hit[:, n_out + 1:], clean[T:T + 7, n_out + 1:])
    else:
        v, c = got.view(torch.bfloat16), clean.view(torch.bfloat16)
        assert v[5].isnan().all()
        others = [f for f in range(n_out) if f != 9]
        assert torch.equal(v[T:T + 7][:, others], c[T:T + 7][:, others])
        assert not v[T:T + 7, 9].isfinite().any()


@pytest.mark.parametrize("bad", [-3, 18])
def test_product_bad_count_is_reported_and_clamped(L, bad):
    R, T, E = 1, 17, 2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, xv = make_rows(L, E * R * T, 64, "bf16", 1)
    w, wv = make_rows(L, E * 64, 64, "bf16", 2)
    y = torch.zeros(E * R * T + 1, 64, dtype=torch.bfloat16, device="cuda")
    bs = L.geometry(T, R, E, err=err)
    c = torch.tensor([[2], [bad]], dtype=torch.int64, device="cuda")
    L.llmoe_expert_product(x, w, y[:-1], c, 64, 64, 0, 0, 0, bs)
    assert L.llmoe_get_error(bs) == L.LLMOE_DEV_SLOT_RANGE
    clamped = np.array([[2], [min(max(bad, 0), T)]])
    at, v, e = ref.product(xv, wv.reshape(E, 64, 64), clamped, T, False)
    close(wide(y)[at], v, e, "bf16")
    rest = np.ones(len(y), bool)
    rest[at] = False
    assert not wide(y)[rest].any()


@pytest.mark.parametrize("dtype", ["bf16", "mx8"])
def test_product_most_experts(L, dtype):
    R, T, E = 1, 1, 8192
    c = (np.random.RandomState(3).rand(E, 1) < 0.3).astype(np.int64)
    check_product(L, R, T, E, 32, 32, dtype, "bf16", dtype == "mx8", c)


@pytest.mark.parametrize("n_in,n_out", [(4096, 64), (64, 4096)])
def test_product_offsets_past_32_bits(L, n_in, n_out):
    """x or y larger than 4 GiB, rows received at the very end of it."""
    R, T, E = 1, 80000, 8
    rows = E * R * T
    counts = np.array([[2], [0], [0], [0], [0], [0], [0], [T]], np.int64)
    counts[3] = 5
    used = np.concatenate([np.arange(2), np.arange(3 * T, 3 * T + 5), np.arange(rows - 3, rows)])
    g = rnd(5)
    x = torch.zeros(rows, n_in, dtype=torch.bfloat16, device="cuda")
    xv = torch.randn(len(used), n_in, generator=g).bfloat16()
    x[torch.from_numpy(used).cuda()] = xv.cuda()
    w = (torch.randn(E, n_out, n_in, generator=g) * n_in ** -0.5).bfloat16()
    y = torch.zeros(rows, n_out, dtype=torch.bfloat16, device="cuda")
    L.llmoe_expert_product(x, w.cuda(), y, torch.from_numpy(counts).cuda(), n_in, n_out, 0, 0, 0, L.geometry(T, R, E))
    got = wide(y[torch.from_numpy(used).cuda()])
    for i, r in enumerate(used):
        a, b = wide(xv)[i], wide(w)[r // T]
        close(got[i], b @ a, n_in * 2.0 ** -23 * (np.abs(b) @ np.abs(a)), "bf16")
    assert not bool(y[2:3 * T].any()) and not bool(y[3 * T + 5:7 * T].any())
    del x, y
    torch.cuda.empty_cache()


def test_norm_offsets_past_32_bits(L):
    rows, hidden = 300000, 7168  # 4.3 GB
    x = torch.ones(rows, hidden, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(3, hidden, generator=rnd(2)).bfloat16()
    x[-3:] = last.cuda()
    w = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    L.llmoe_add_rmsnorm(x, None, w, 0.0, None, x, rows, hidden, 0, 0)
    v = ref.rmsnorm(wide(last), np.ones(hidden), 0.0)
    close(wide(x[-3:]), v, np.abs(v) * NORM_ERR, "bf16")
    assert bool((x[:-3] == 1).all())
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "mx8"])
def test_product_many_calls(L, dtype):
    """Calls with cold caches, warm ones and after other kernels: the same bits
    every time and no wait that expires."""
    R, T, E, K, n_in, n_out = 1, 128, 256, 8, 2048, 512
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bs = L.geometry(T, R, E, err=err)
    code = L.ROW_DTYPE_CODES
    g = rnd(31)
    x, _ = make_rows(L, E * R * T // 64, n_in, dtype, 1)
    x = x.repeat(64, 1)
    w, _ = make_rows(L, 64 * 2 * n_out, n_in, dtype, 2, 0.05)
    w = w.repeat(4, 1)
    flush = torch.empty(64 << 20, dtype=torch.float32, device="cuda")
    for _ in range(6):
        counts = torch.zeros(E, R, dtype=torch.int64)
        counts[torch.randperm(E, generator=g)[:K]] = 1
        c = counts.cuda()
        first = None
        for call in range(40):
            y = torch.zeros(E * R * T, n_out, dtype=torch.bfloat16, device="cuda")
            if call % 4 == 1:
                flush.add_(1)
            L.llmoe_expert_product(x, w, y, c, n_in, n_out, code[dtype], 0, L.LLMOE_PRODUCT_SWIGLU, bs)
            first = y if first is None else first
            assert torch.equal(first, y)
        assert int(err) == 0
        assert int(first.any(1).sum()) == K


@pytest.mark.parametrize("dtype", ["bf16", "mx8"])
def test_product_of_tensors_16_bytes_off(L, dtype):
    """Every pointer 16-byte aligned and no more."""
    R, T, E, n_in, n_out = 2, 11, 4, 160, 96
    counts = some_counts(E, R, T, "ragged", 8)
    x, xv = make_rows(L, E * R * T, n_in, dtype, 1)
    w, wv = make_rows(L, E * n_out, n_in, dtype, 2, 0.1)
    shift = lambda t: torch.cat([torch.zeros(16, dtype=torch.uint8, device="cuda"), t.reshape(-1).view(torch.uint8)])[16:]
    y = torch.zeros(16 + E * R * T * n_out * 2, dtype=torch.uint8, device="cuda")[16:]
    L.llmoe_expert_product(shift(x), shift(w), y, torch.from_numpy(counts).cuda(), n_in, n_out,
                           L.ROW_DTYPE_CODES[dtype], 0, 0, L.geometry(T, R, E))
    at, v, err = ref.product(xv, wv.reshape(E, n_out, n_in), counts, T, False)
    close(wide(y.view(torch.bfloat16).reshape(-1, n_out))[at], v, err, "bf16")


def test_products_on_two_streams_at_once(L):
    """Two calls in flight, each with every SM in its grid."""
    R, T, E, n = 2, 200, 8, 512
    c = torch.from_numpy(some_counts(E, R, T, "ragged", 6)).cuda()
    bs = L.geometry(T, R, E)
    sets = []
    for dtype in ("bf16", "mx8"):
        x, _ = make_rows(L, E * R * T, n, dtype, 3)
        w, _ = make_rows(L, E * n, n, dtype, 4, 0.05)
        ys = [torch.zeros(E * R * T, n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        sets.append((x, w, ys, L.ROW_DTYPE_CODES[dtype], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for x, w, ys, code, _ in sets:
        L.llmoe_expert_product(x, w, ys[0], c, n, n, code, 0, 0, bs)
    torch.cuda.synchronize()
    for _ in range(5):
        for x, w, ys, code, s in sets:
            L.llmoe_expert_product(x, w, ys[1], c, n, n, code, 0, 0, bs, s)
    torch.cuda.synchronize()
    for _, _, ys, _, _ in sets:
        assert torch.equal(ys[0], ys[1]) and bool(ys[0].any())


# ---------------------------------------------------------------------------
# one MoE block: norm, router, dispatch, products, combine
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "mx8"])
def test_counts_from_the_rank_buffers(L, dtype):
    """The product driven by a dispatch's own count words (counts NULL)."""
    R, T, E, K, n_in, n_out = 2, 9, 6, 2, 512, 64
    code = L.ROW_DTYPE_CODES
    rb_in = L.llmoe_row_bytes(n_in, code[dtype])
    x, _ = make_rows(L, R * T, n_in, dtype, 3)
    w, _ = make_rows(L, E * n_out, n_in, dtype, 4, 0.05)
    idx = torch.rand(R, T, E, generator=rnd(1)).argsort(-1)[..., :K].contiguous()
    idx[0, 3, 1] = -1
    rb = L.RankBuffers(T, rb_in // 2, R, E, fill=0xA5)
    recv = torch.zeros(E * R * T, rb_in, dtype=torch.uint8, device="cuda")
    src = torch.zeros(E * R * T, dtype=torch.int32, device="cuda")
    for s in (0, 1):
        bs = rb.buf_set(s, K)
        L.llmoe_clean(bs)
        L.llmoe_dispatch_unpack(x.view(torch.uint8).view(torch.bfloat16), idx.cuda(), recv.view(torch.bfloat16), src, bs)
        counts = torch.empty(E, R, dtype=torch.int64, device="cuda")
        slot = torch.empty(R, T, K, dtype=torch.int32, device="cuda")
        L.llmoe_route(idx.cuda(), slot, counts, bs)
        ya, yb = (torch.zeros(E * R * T, n_out, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        L.llmoe_expert_product(recv, w, ya, None, n_in, n_out, code[dtype], 0, 0, bs)
        L.llmoe_expert_product(recv, w, yb, counts, n_in, n_out, code[dtype], 0, 0, L.geometry(T, R, E))
        assert torch.equal(ya, yb) and bool(ya.any())


@pytest.mark.parametrize("rows,dtype", [("same", "bf16"), ("same", "fp16"), ("mx8", "bf16")])
def test_moe_block(L, rows, dtype):
    """The whole block against its definition, given the block's own choice of
    experts (checked against the router's definition from its own logits)."""
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    R, T, n, H, I, E, K = 2, 24, 19, 512, 160, 8, 3
    t, g = TORCH[dtype], rnd(12)
    norm_w = (1 + 0.1 * torch.randn(H, generator=g)).to(t)
    router_w = (torch.randn(E, H, generator=g) * H ** -0.5).to(t)
    gate_up = (torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).to(t)
    down = (torch.randn(E, H, I, generator=g) * I ** -0.5).to(t)
    bias = torch.randint(-2, 3, (E,), generator=g).float() / 8
    x = torch.randn(R, n, H, generator=g).to(t)
    res = torch.randn(R, n, H, generator=g).to(t)
    active = (torch.rand(R, n, generator=g) < 0.85).to(torch.uint8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = MoEBlock(T, R, K, norm_w.cuda(), router_w.cuda(), gate_up.cuda(), down.cuda(), bias.cuda(), dtype, rows,
                 scale=2.0, err=err)
    residual, out = res.cuda(), torch.full((R, n, H), float("nan"), dtype=t, device="cuda")
    m.forward(x.cuda(), residual, out, active.cuda())
    first = out.clone()
    h = (x.float() + res.float()).to(t)
    assert torch.equal(residual.cpu(), h)
    # again on the same buffers, without and within a CUDA graph: the same bits
    residual.copy_(res.cuda())
    m.forward(x.cuda(), residual, out, active.cuda())
    assert torch.equal(out, first)
    xs, acts = x.cuda(), active.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(xs, residual, out, acts)
    residual.copy_(res.cuda())
    out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and int(err) == 0

    tokens = R * n
    v = ref.rmsnorm(wide(h).reshape(tokens, H), wide(norm_w), 1e-6)
    xn = wide(m.xn)[:tokens]
    close(xn, v, np.abs(v) * NORM_ERR, dtype)
    logits = m.logits[:tokens].cpu()
    want = xn @ wide(router_w).T
    assert (np.abs(logits.double().numpy() - want) <= H * 2.0 ** -23 * (np.abs(xn) @ np.abs(wide(router_w)).T)).all()
    idx, w, gap = ref.router(logits.numpy(), bias.numpy(), active.reshape(-1).numpy(), K, "sigmoid", True, 2.0)
    assert gap > 1e-6
    assert np.array_equal(m.topk_idx[:tokens].cpu().numpy(), idx)
    # the experts on the rows that were dispatched, in 64 bits, each rounding of the path bounded
    if rows == "mx8":
        xe = ref.mx8_values(m.rows.cpu().numpy()[:tokens], H)
        gu = ref.mx8_values(m.gate_up.cpu().numpy(), H)
        dn = ref.mx8_values(m.down.cpu().numpy(), I)
    else:
        xe, gu, dn = xn, wide(gate_up), wide(down)
    step = 2.0 ** -4 if rows == "mx8" else HALF_ULP[dtype]  # h's rounding, relative to its group's largest value
    got = wide(first).reshape(tokens, H)
    topk_w = m.topk_w[:tokens].cpu().double().numpy()
    for i in range(tokens):
        total, tol = np.zeros(H), np.zeros(H)
        for k in range(K):
            e = idx[i, k]
            if e < 0:
                continue
            _, hv, he = ref.product(xe[i:i + 1], gu[e:e + 1], np.array([[1]]), 1, True)
            hv, he = hv[0], he[0]
            he = he + step * (np.repeat(np.abs(hv).reshape(-1, 32).max(1), 32) if rows == "mx8" else np.abs(hv)) + TINY[dtype]
            y = dn[e] @ hv
            ye = np.abs(dn[e]) @ he + I * 2.0 ** -23 * (np.abs(dn[e]) @ np.abs(hv))
            ye += (np.abs(y) + ye) * HALF_ULP[dtype] + TINY[dtype]
            total += topk_w[i, k] * y
            tol += topk_w[i, k] * ye
        tol += (np.abs(total) + tol) * (HALF_ULP[dtype] + K * 2.0 ** -23) + TINY[dtype]
        assert (np.abs(got[i] - total) <= tol).all(), i


def test_moe_block_refuses_too_many_tokens(L):
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    m = MoEBlock(4, 2, 1, z(64), z(2, 64), z(2, 64, 64), z(2, 64, 32))
    with pytest.raises(ValueError):
        m.forward(z(2, 5, 64), z(2, 5, 64), z(2, 5, 64))


@pytest.mark.parametrize("call", ["route", "dispatch", "dispatch_unpack", "combine", "combine_staged"])
def test_router_queued_before(L, call):
    """A call queued right behind the router that writes its topk_idx and
    topk_w, all launched while the device is still busy, reads what the router
    wrote: the same bytes as with a synchronize between the two."""
    R, T, H, E, K = 4, 48, 512, 32, 4
    logits = torch.randn(R * T, E, generator=rnd(77)).cuda()
    x = torch.randn(R, T, H, generator=rnd(78)).to(torch.bfloat16).cuda()
    y = torch.randn(E, R, T, H, generator=rnd(79)).to(torch.bfloat16).cuda()
    idx = torch.empty(R, T, K, dtype=torch.int64, device="cuda")
    w = torch.empty(R, T, K, dtype=torch.float32, device="cuda")

    def run(between):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        rb = L.RankBuffers(T, H, R, E, fill=0)
        s = 1 if call.startswith("combine") else 0
        bs = rb.buf_set(s, K, err=err)
        recv_x = torch.zeros(E, R, T, H, dtype=torch.bfloat16, device="cuda")
        recv_src = torch.zeros(E, R, T, dtype=torch.int32, device="cuda")
        out = torch.zeros(R, T, H, dtype=torch.bfloat16, device="cuda")
        slot = torch.zeros(R, T, K, dtype=torch.int32, device="cuda")
        counts = torch.zeros(E, R, dtype=torch.int64, device="cuda")
        idx.fill_(-1)
        w.fill_(0)
        torch.cuda.synchronize()
        torch.cuda._sleep(4_000_000)
        L.llmoe_topk_router(logits, None, None, idx, w, R * T, E, K, L.LLMOE_DTYPE_FP32, L.LLMOE_SCORE_SOFTMAX, 0, 1.0)
        between()
        if call == "route":
            L.llmoe_route(idx, slot, counts, bs)
        elif call == "dispatch":
            L.llmoe_dispatch(x, idx, bs)
        elif call == "dispatch_unpack":
            L.llmoe_dispatch_unpack(x, idx, recv_x, recv_src, bs)
        elif call == "combine":
            L.llmoe_combine(y, idx, w, out, bs)
        else:
            L.llmoe_combine_staged(y, idx, w, out, bs)
        torch.cuda.synchronize()
        assert int(err) == 0
        return rb.storage, recv_x, recv_src, out, slot, counts

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        for got, ref_ in zip(run(lambda: None), want):
            assert torch.equal(got, ref_)


@pytest.mark.parametrize("rows", ["same", "mx8"])
def test_moe_block_queued(L, rows):
    """A block's calls all queued while the device is still busy, over buffers
    that held something else: the bits of a call on an idle device."""
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    R, T, n, H, I, E, K = 4, 64, 37, 1536, 768, 32, 4
    g = rnd(91)
    new = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(torch.bfloat16).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = MoEBlock(T, R, K, torch.ones(H, dtype=torch.bfloat16, device="cuda"), new(E, H), new(E, 2 * I, H), new(E, H, I),
                 None, "bf16", rows, err=err)
    x, res0 = H ** 0.5 * new(R, n, H), new(R, n, H)
    out, outs = torch.empty_like(x), []
    res = res0.clone()
    for busy in (False, True, True):
        res.copy_(res0)
        out.zero_()
        m.topk_idx.fill_(-1)
        m.topk_w.zero_()
        m.logits.zero_()
        m.recv_x.zero_()
        m.recv_src.zero_()
        torch.cuda.synchronize()
        if busy:
            torch.cuda._sleep(8_000_000)
        m.forward(x, res, out)
        torch.cuda.synchronize()
        assert int(err) == 0
        outs.append(out.clone())
    assert torch.isfinite(outs[0]).all() and (outs[0] != 0).any()
    assert torch.equal(outs[1], outs[0]) and torch.equal(outs[2], outs[0])


@pytest.mark.parametrize("between", ["pack", "norm", "product"])
def test_router_before_an_early_combine(L, between):
    """LLMOE_FLAG_INPUTS_READY on a combine with one other call between the
    router and it, all queued while the device is busy: the combine may read
    topk_idx and topk_w before its wait, and they are there."""
    R, T, H, E, K = 1, 1, 512, 8192, 8
    logits = torch.randn(1, E, generator=rnd(81)).cuda()
    y = torch.randn(E, R, T, H, generator=rnd(82)).to(torch.bfloat16).cuda()
    z = torch.randn(32, 64, generator=rnd(83)).to(torch.bfloat16).cuda()
    w1, counts = torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.ones(1, dtype=torch.int64, device="cuda")
    packed = torch.empty(32, 80, dtype=torch.uint8, device="cuda")
    zz, prod = torch.empty_like(z), torch.empty(1, 32, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(R, T, K, dtype=torch.int64, device="cuda")
    w = torch.empty(R, T, K, dtype=torch.float32, device="cuda")
    out = torch.empty(R, T, H, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rb = L.RankBuffers(T, H, R, E, fill=0)
    one = L.geometry(1, 1, 1, err)
    outs = []
    for sync in (True, False, False, False):
        idx.fill_(-1)
        w.zero_()
        out.zero_()
        rb.storage.zero_()
        torch.cuda.synchronize()
        torch.cuda._sleep(4_000_000)
        L.llmoe_topk_router(logits, None, None, idx, w, 1, E, K, L.LLMOE_DTYPE_FP32, L.LLMOE_SCORE_SOFTMAX, 0, 1.0)
        if between == "pack":
            L.llmoe_pack_mx8(z, packed, 32, 64, L.LLMOE_DTYPE_BF16)
        elif between == "norm":
            L.llmoe_add_rmsnorm(z, None, w1, 1e-6, None, zz, 32, 64, L.LLMOE_DTYPE_BF16, L.LLMOE_DTYPE_BF16)
        else:
            L.llmoe_expert_product(z[:1], z, prod, counts, 64, 32, L.LLMOE_DTYPE_BF16, L.LLMOE_DTYPE_BF16, 0, one)
        if sync:
            torch.cuda.synchronize()
        L.llmoe_combine(y, idx, w, out, rb.buf_set(1, K, err=err, flags=L.LLMOE_FLAG_INPUTS_READY))
        torch.cuda.synchronize()
        assert int(err) == 0
        outs.append(out.clone())
    assert (outs[0] != 0).any()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("rows", ["same", "mx8"])
def test_moe_block_changing_inputs(L, rows):
    """Two inputs in turn through one block's buffers, all queued: each has the
    bits of a call on an idle device, so no step reads what the other left."""
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    R, T, H, I, E, K = 2, 32, 512, 128, 8, 2
    g = rnd(95)
    new = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(torch.bfloat16).cuda()
    m = MoEBlock(T, R, K, torch.ones(H, dtype=torch.bfloat16, device="cuda"), new(E, H), new(E, 2 * I, H), new(E, H, I),
                 None, "bf16", rows)
    xs = [new(R, T, H), 8 * new(R, T, H)]
    res, outs = [torch.zeros_like(x) for x in xs], [torch.empty_like(x) for x in xs]
    want = []
    for x, r, o in zip(xs, res, outs):
        m.forward(x, r, o)
        torch.cuda.synchronize()
        want.append(o.clone())
    assert not torch.equal(want[0], want[1])
    for _ in range(5):
        torch.cuda._sleep(4_000_000)
        for _ in range(8):
            for x, r, o in zip(xs, res, outs):
                r.zero_()
                m.forward(x, r, o)
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
