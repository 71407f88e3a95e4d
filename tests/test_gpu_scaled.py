"""GPU tests of the block-scaled operators (FP8B rows and weights, their product)
and of the router with groups, against their definitions in 64 bits
(tests/fp8b_reference.py).

Tolerances, derived from the arithmetic each call documents:
- packing is exact: one fp32 division, one reciprocal, one product, one rounding
  to e4m3, each of which rounds to nearest;
- the fp32 norm before it: 48 roundings of 2^-24 (test_gpu_block.py), 3e-6;
- products: an fp32 sum of n products, each addition within 2^-23 of the sum of
  the magnitudes (the tensor cores truncate), the two scales of a block and its
  addition two roundings and one more addition (fp8b_reference.product_error),
  and the rounding to the output type;
- router weights: exponential, sum and division, one rounding each per term.
"""
import numpy as np
import pytest
import torch

import block_reference as ref
import fp8b_reference as fp8b

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
    tol = err + (np.abs(want) + err) * HALF_ULP[dtype] + TINY[dtype]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.abs(got - want)[bad][:4], tol[bad][:4])


# ---------------------------------------------------------------------------
# rows and weights
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,hidden", [(1, 16), (3, 48), (2, 128), (5, 144), (9, 528), (4, 7168), (3, 2000),
                                         (700, 272), (5000, 96), (2, 32768)])
def test_pack_rows_is_exact(L, rows, hidden, dtype):
    g = rnd(rows + hidden)
    size = torch.exp2(torch.randint(-6, 7, (rows, fp8b.blocks(hidden), 1), generator=g).float()).expand(-1, -1, 128)
    x = (torch.randn(rows, hidden, generator=g) * size.reshape(rows, -1)[:, :hidden]).to(TORCH[dtype])
    x[0, :128] = 0  # a block of zeros
    if hidden >= 528:
        x[0, 128:256] = 0
        x[0, 128:132] = torch.tensor([448.0, 17.0, 19.0, 0.0009765625])  # scale 1: midpoints of codes, a half of the least
        x[0, 256:384] = 0
        x[0, 256] = torch.finfo(TORCH[dtype]).max
        x[0, 384:512] = 0
        x[0, 384] = torch.finfo(TORCH[dtype]).tiny  # its scale is the least one
    got = torch.full((rows * fp8b.row_bytes(hidden) + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    assert L.llmoe_row_bytes(hidden, L.LLMOE_DTYPE_FP8B) == fp8b.row_bytes(hidden)
    L.llmoe_pack_fp8b(x.cuda(), got[:-16], rows, hidden, L.ROW_DTYPE_CODES[dtype])
    assert (got[-16:] == 0xA5).all()
    got = got[:-16].reshape(rows, -1).cpu().numpy()
    want = fp8b.pack(x.float().numpy())
    assert np.array_equal(got[:, hidden:], want[:, hidden:])
    assert np.array_equal(ref.E4M3[got[:, :hidden]], ref.E4M3[want[:, :hidden]])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,hidden", [(1, 64), (3, 96), (5, 2048), (2, 7168), (1, 32768), (700, 224), (410, 7168),
                                         (1300, 2096), (153, 16384), (160, 32768), (2048, 16)])
def test_add_rmsnorm(L, rows, hidden, dtype):
    g = rnd(rows * 7 + hidden)
    x = torch.randn(rows, hidden, generator=g).to(TORCH[dtype])
    res = (3 * torch.randn(rows, hidden, generator=g)).to(TORCH[dtype])
    w = (1 + 0.2 * torch.randn(hidden, generator=g)).to(TORCH[dtype])
    x[rows // 2] = 0
    if rows > 1:
        res[0] = -x[0]  # eps alone under the root
    h = (x.float() + res.float()).to(TORCH[dtype])
    rb = fp8b.row_bytes(hidden)
    got = torch.full((rows * rb + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    hout = torch.empty_like(x, device="cuda")
    L.llmoe_add_rmsnorm(x.cuda(), res.cuda(), w.cuda(), 1e-5, hout, got[:-16], rows, hidden, L.DTYPE_CODES[dtype],
                        L.LLMOE_DTYPE_FP8B)
    assert torch.equal(hout.cpu(), h)
    assert (got[-16:] == 0xA5).all()
    v = ref.rmsnorm(wide(h), wide(w), 1e-5)
    fp8b.check(got[:-16].reshape(rows, rb).cpu().numpy(), v, np.abs(v) * NORM_ERR)


def test_pack_of_nan_and_infinity(L):
    x = torch.ones(1, 400, dtype=torch.bfloat16)
    x[0, 5], x[0, 399] = float("nan"), float("-inf")
    got = torch.empty(1, 416, dtype=torch.uint8, device="cuda")
    L.llmoe_pack_fp8b(x.cuda(), got, 1, 400, L.LLMOE_DTYPE_BF16)
    q, s, pad = fp8b.split(got.cpu().numpy(), 400)
    assert np.isnan(s[0, [0, 3]]).all() and (s[0, 1:3] == np.float32(1) / np.float32(448)).all() and not pad.any()
    assert np.isnan(q[0, :128]).all() and (q[0, 128:384] == 448).all() and np.isnan(q[0, 384:]).all()
    w = torch.ones(2, 140, 144, dtype=torch.float32)
    w[0, 3, 130] = float("inf")
    w[1, 139, 0] = float("nan")
    codes = torch.empty(2, 140, 144, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2, 2, 2, device="cuda")
    L.llmoe_pack_fp8b_weights(w.cuda(), codes, scales, 2, 140, 144, L.LLMOE_DTYPE_FP32)
    bad = torch.zeros(2, 2, 2, dtype=torch.bool)
    bad[0, 0, 1] = bad[1, 1, 0] = True
    assert torch.equal(scales.cpu().isnan(), bad)
    v = codes.cpu().view(torch.float8_e4m3fn).float()
    assert v[0, :128, 128:].isnan().all() and (v[0, :, :128] == 448).all() and (v[0, 128:] == 448).all()
    assert v[1, 128:, :128].isnan().all() and (v[1, :128] == 448).all() and (v[1, :, 128:] == 448).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("matrices,rows,cols", [(1, 1, 16), (3, 128, 128), (2, 129, 144), (5, 40, 272), (1, 2000, 1040),
                                                (40, 256, 512), (300, 8, 48)])
def test_pack_weights_is_exact(L, matrices, rows, cols, dtype):
    g = rnd(matrices + rows + cols)
    w = torch.randn(matrices, rows, cols, generator=g).to(TORCH[dtype])
    w[0, :128, :128] = 0  # a block of zeros
    codes = torch.full((w.numel() + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    n = matrices * fp8b.blocks(rows) * fp8b.blocks(cols)
    scales = torch.full((n + 4,), -1.0, device="cuda")
    L.llmoe_pack_fp8b_weights(w.cuda(), codes[:-16], scales[:-4], matrices, rows, cols, L.DTYPE_CODES[dtype])
    assert (codes[-16:] == 0xA5).all() and (scales[-4:] == -1).all()
    want, s = fp8b.pack_weights(w.float().numpy())
    assert np.array_equal(scales[:-4].cpu().numpy(), s.reshape(-1))
    assert np.array_equal(ref.E4M3[codes[:-16].cpu().numpy()], ref.E4M3[want.reshape(-1)])


def test_pack_offsets_past_32_bits(L):
    """A matrix, and rows, of more than 4 GiB: their last values."""
    rows, cols = 360448, 8192  # 5.9 GB
    w = torch.zeros(1, rows, cols, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(160, cols, generator=rnd(4)).bfloat16()
    w[0, -160:] = last.cuda()
    codes = torch.empty(1, rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(1, rows // 128, cols // 128, device="cuda")
    L.llmoe_pack_fp8b_weights(w, codes, scales, 1, rows, cols, L.LLMOE_DTYPE_BF16)
    want, s = fp8b.pack_weights(torch.cat([torch.zeros(96, cols), last.float()]).numpy())
    assert np.array_equal(scales[0, -2:].cpu().numpy(), s)
    assert np.array_equal(ref.E4M3[codes[0, -256:].cpu().numpy()], ref.E4M3[want])
    assert not bool(codes[0, :-256].any())
    del codes
    out = torch.empty(rows, fp8b.row_bytes(cols), dtype=torch.uint8, device="cuda")
    L.llmoe_pack_fp8b(w[0], out, rows, cols, L.LLMOE_DTYPE_BF16)
    want = fp8b.pack(last.float().numpy())
    got = out[-160:].cpu().numpy()
    assert np.array_equal(got[:, cols:], want[:, cols:])
    assert np.array_equal(ref.E4M3[got[:, :cols]], ref.E4M3[want[:, :cols]])
    del w, out
    torch.cuda.empty_cache()


def test_nothing_to_pack(L):
    L.llmoe_pack_fp8b(None, None, 0, 64, 0)
    L.llmoe_pack_fp8b_weights(None, None, None, 0, 64, 64, 0)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# router with groups
# ---------------------------------------------------------------------------

def route(L, logits, bias, active, K, groups, kept, top2, dtype, scoring, renorm, scale):
    rows, E = logits.shape
    idx = torch.full((rows + 1, K), -7, dtype=torch.int64, device="cuda")
    w = torch.full((rows + 1, K), -7.0, device="cuda")
    flags = (L.LLMOE_ROUTER_RENORM if renorm else 0) | (L.LLMOE_ROUTER_GROUP_TOP2 if top2 else 0)
    L.llmoe_group_router(logits.cuda(), None if bias is None else bias.cuda(), None if active is None else active.cuda(),
                         idx[:rows], w[:rows], rows, E, K, groups, kept, L.DTYPE_CODES[dtype],
                         L.LLMOE_SCORE_SIGMOID if scoring == "sigmoid" else L.LLMOE_SCORE_SOFTMAX, flags, scale)
    assert (idx[rows] == -7).all() and (w[rows] == -7).all()
    return idx[:rows].cpu().numpy(), w[:rows].cpu().numpy().astype(np.float64)


GROUP_SHAPES = [  # rows, E, K, groups, kept
    (1, 256, 8, 8, 4), (300, 256, 8, 8, 4), (70, 160, 6, 8, 3), (33, 64, 6, 8, 1), (40, 128, 8, 4, 3), (9, 512, 32, 16, 5),
    (21, 60, 5, 5, 2), (13, 96, 3, 3, 1), (17, 7, 3, 7, 4), (50, 8, 2, 2, 1), (5, 1, 1, 1, 1), (12, 384, 8, 1, 1),
    (30, 72, 4, 36, 7), (6, 512, 6, 256, 3), (8, 640, 8, 10, 4), (4, 2048, 8, 32, 8), (3, 8192, 32, 256, 2),
    (2, 8190, 9, 45, 44), (40, 352, 8, 11, 6), (40, 32, 4, 4, 2), (40, 480, 8, 16, 9), (25, 288, 8, 8, 4)]


@pytest.mark.parametrize("scoring,top2", [("sigmoid", True), ("sigmoid", False), ("softmax", False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,E,K,groups,kept", GROUP_SHAPES)
def test_group_router(L, rows, E, K, groups, kept, dtype, scoring, top2):
    g = rnd(rows * 31 + E + groups)
    logits = torch.randint(-24, 25, (rows, E), generator=g).float() / 8  # exact in every type; many ties
    b = torch.randint(-1, 2, (E,), generator=g).float() / 4 if rows % 2 else None
    active = (torch.rand(rows, generator=g) < 0.8).to(torch.uint8) if rows > 4 else None
    renorm = rows % 3 != 0
    gi, gw = route(L, logits.to(TORCH[dtype]), b, active, K, groups, kept, top2, dtype, scoring, renorm, 2.5)
    seen = 0
    for r in range(rows):
        idx, w, gap = fp8b.group_router(logits[r:r + 1].numpy(), None if b is None else b.numpy(),
                                        None if active is None else active[r:r + 1].numpy(), K, groups, kept, top2,
                                        scoring, renorm, 2.5)
        if gap < 4e-6:  # fp32 keys (sums of two, below 4: 2^-22 each rounding) need not order as the exact ones
            continue
        seen += 1
        assert np.array_equal(gi[r], idx[0]), r
        assert (np.abs(gw[r] - w[0]) <= w[0] * (E / 32 + K + 32) * 2.0 ** -23).all()
    assert seen > rows * 0.7 or rows < 10


@pytest.mark.parametrize("scoring,top2", [("sigmoid", True), ("softmax", False)])
@pytest.mark.parametrize("E,K,groups,kept,spread", [(256, 8, 8, 4, 1.0), (256, 8, 8, 4, 12.0), (160, 6, 8, 3, 3.0),
                                                    (512, 32, 16, 8, 1.0)])
def test_group_router_continuous_logits(L, E, K, groups, kept, spread, scoring, top2):
    rows = 300
    g = rnd(E + K)
    logits, b = torch.randn(rows, E, generator=g) * spread, torch.randn(E, generator=g) * 0.3
    gi, gw = route(L, logits, b, None, K, groups, kept, top2, "fp32", scoring, True, 1.0)
    seen = 0
    for r in range(rows):
        idx, w, gap = fp8b.group_router(logits[r:r + 1].numpy(), b.numpy(), None, K, groups, kept, top2, scoring, True, 1.0)
        if gap < 1e-5 * max(1.0, spread):
            continue
        seen += 1
        assert np.array_equal(gi[r], idx[0]), r
        assert (np.abs(gw[r] - w[0]) <= w[0] * (E / 32 + K + 32 + 2 * np.abs(logits[r].numpy()).max()) * 2.0 ** -23).all()
    assert seen > rows // 2


@pytest.mark.parametrize("E,K", [(256, 8), (160, 6), (33, 4), (512, 32), (1024, 8)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_one_group_is_the_plain_router(L, E, K, scoring):
    """Also with every group kept: llmoe_topk_router's own choices, bit for bit."""
    rows = 200
    logits, b = torch.randn(rows, E, generator=rnd(E)), 0.2 * torch.randn(E, generator=rnd(K))
    code = L.LLMOE_SCORE_SIGMOID if scoring == "sigmoid" else L.LLMOE_SCORE_SOFTMAX
    for renorm in (False, True):
        idx = torch.empty(rows, K, dtype=torch.int64, device="cuda")
        w = torch.empty(rows, K, device="cuda")
        L.llmoe_topk_router(logits.cuda(), b.cuda(), None, idx, w, rows, E, K, L.LLMOE_DTYPE_FP32, code, int(renorm), 2.5)
        for groups in {1, 8 if E % 8 == 0 else 3}:
            gi, gw = route(L, logits, b, None, K, groups, groups, False, "fp32", scoring, renorm, 2.5)
            assert np.array_equal(gi, idx.cpu().numpy())
            assert (np.abs(gw - wide(w)) <= wide(w) * (E / 32 + K + 32) * 2.0 ** -23).all()


@pytest.mark.parametrize("E", [40, 256, 1000])
@pytest.mark.parametrize("scoring,top2", [("sigmoid", True), ("sigmoid", False), ("softmax", False)])
def test_group_router_masked_experts(L, E, scoring, top2):
    inf, nan = float("inf"), float("nan")
    K, G, kept = 4, 8 if E % 8 == 0 else 4, 2
    S = E // G
    logits = torch.zeros(10, E)
    logits[0] = -inf  # nothing can be chosen
    logits[1] = -inf
    logits[1, 0], logits[1, E - 1] = 0.5, 1.5  # one expert of two groups
    logits[2] = nan
    logits[2, 3] = -2.0
    logits[3, S:] = nan  # all but the first group
    logits[4, 1] = logits[4, E - 2] = inf  # two of the largest
    logits[5] = torch.finfo(torch.float32).min  # a mask of the type's lowest value, over the whole row
    logits[6, :S] = 2.0  # the best group, but for one expert masked
    logits[6, 1:S] = -inf
    logits[7, 2 * S] = 3.0  # the single best expert, in a group that ties otherwise
    logits[8, S:2 * S] = logits[8, 3 * S:4 * S] = 1.0  # equal groups: the lower ones
    logits[8, 2 * S:3 * S] = 1.0
    logits[9] = torch.finfo(torch.float32).max
    bias = torch.zeros(E)
    bias[2] = -inf  # masked by the bias
    for b in (None, bias):
        idx, w, _ = fp8b.group_router(np.where(np.isnan(logits.numpy()), -np.inf, logits.numpy()),
                                      None if b is None else b.numpy(), None, K, G, kept, top2, scoring, True, 1.0)
        gi, gw = route(L, logits, b, None, K, G, kept, top2, "fp32", scoring, True, 1.0)
        assert np.array_equal(gi, idx)
        assert np.allclose(gw, w, rtol=64 * 2.0 ** -23, atol=0)


@pytest.mark.parametrize("E,K,groups,kept", [(256, 8, 8, 4), (160, 6, 8, 3), (512, 8, 16, 5), (96, 3, 3, 2), (32, 4, 4, 2)])
@pytest.mark.parametrize("top2", [True, False])
def test_group_router_far_logits(L, E, K, groups, kept, top2):
    """Sigmoids near fp32's smallest: still the largest logits', and with their weights.
    Keys a 16th apart differ by 6%; -88.5 has 2^21 of fp32's smallest steps (2^-149),
    so half a step is less than 2^-22 of it."""
    rows = 24
    g = rnd(E + kept)
    logits = torch.stack([torch.randperm(E, generator=g).float() / 16 - 88.5 for _ in range(rows)])
    other = torch.rand(rows, E, generator=g)
    logits[8:16] += (other[8:16] < 0.1) * 60.0  # near ones among them, no sigmoid of them 1
    logits[16:][other[16:] < 0.5] = -float("inf")
    gi, gw = route(L, logits, None, None, K, groups, kept, top2, "fp32", "sigmoid", True, 2.5)
    idx, w, _ = fp8b.group_router(logits.numpy(), None, None, K, groups, kept, top2, "sigmoid", True, 2.5, same=0)
    if top2:  # sums of two keys may be as near as rounding
        same = (gi == idx).all(1)
        assert same.mean() > 0.9
        gi, gw, idx, w = gi[same], gw[same], idx[same], w[same]
    assert np.array_equal(gi, idx)
    assert (np.abs(gw - w) <= w * (K + 32 + 2 * 2) * 2.0 ** -23 + 2.5 * 2.0 ** -149).all()


@pytest.mark.parametrize("E,groups", [(256, 8), (160, 8), (264, 8)])
def test_group_router_bias_not_16_byte_aligned(L, E, groups):
    rows, K = 70, 6
    logits = torch.randint(-24, 25, (rows, E), generator=rnd(E)).float() / 8
    flat = torch.randint(-8, 9, (E + 1,), generator=rnd(1)).float() / 8
    idx = torch.empty(rows, K, dtype=torch.int64, device="cuda")
    w = torch.empty(rows, K, device="cuda")
    L.llmoe_group_router(logits.cuda(), flat.cuda()[1:], None, idx, w, rows, E, K, groups, 3, L.LLMOE_DTYPE_FP32,
                         L.LLMOE_SCORE_SOFTMAX, 0, 1.0)
    want, ww, _ = fp8b.group_router(logits.numpy(), flat[1:].numpy(), None, K, groups, 3, False, "softmax", False, 1.0)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert (np.abs(wide(w) - ww) <= ww * (E / 32 + K + 32) * 2.0 ** -23).all()


@pytest.mark.parametrize("E,groups", [(256, 8), (100, 5), (264, 8), (768, 8)])
def test_group_router_logits_not_16_byte_aligned(L, E, groups):
    rows, K = 70, 6
    flat = torch.randint(-24, 25, (rows * E + 1,), generator=rnd(E)).float() / 8
    at = flat.cuda()[1:]
    idx = torch.empty(rows, K, dtype=torch.int64, device="cuda")
    w = torch.empty(rows, K, device="cuda")
    L.llmoe_group_router(at, None, None, idx, w, rows, E, K, groups, 3, L.LLMOE_DTYPE_FP32, L.LLMOE_SCORE_SOFTMAX, 0, 1.0)
    want, ww, _ = fp8b.group_router(flat[1:].reshape(rows, E).numpy(), None, None, K, groups, 3, False, "softmax", False, 1.0)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert (np.abs(wide(w) - ww) <= ww * (E / 32 + K + 32) * 2.0 ** -23).all()


def test_group_router_no_rows(L):
    L.llmoe_group_router(None, None, None, None, None, 0, 8, 2, 4, 2, L.LLMOE_DTYPE_FP32, 0, 2, 1.0)
    torch.cuda.synchronize()


def test_group_router_captured_and_queued(L):
    """Replayed from a graph behind a kernel that writes its logits, and read by a
    dispatch behind it: what a synchronised call gives."""
    R, T, H, E, K = 4, 48, 512, 64, 4
    src = torch.randn(R * T, E, generator=rnd(7)).cuda()
    logits = torch.zeros_like(src)
    x = torch.randn(R, T, H, generator=rnd(8)).bfloat16().cuda()
    idx = torch.empty(R, T, K, dtype=torch.int64, device="cuda")
    w = torch.empty(R, T, K, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rb = L.RankBuffers(T, H, R, E, fill=0)
    bs = rb.buf_set(0, K, err=err)

    def call(sync):
        logits.copy_(src)
        L.llmoe_clean(bs)
        L.llmoe_group_router(logits, None, None, idx, w, R * T, E, K, 8, 3, L.LLMOE_DTYPE_FP32, 0, 3, 1.0)
        if sync:
            torch.cuda.synchronize()
        L.llmoe_dispatch(x, idx, bs)

    call(True)
    torch.cuda.synchronize()
    want = idx.clone(), w.clone(), rb.storage.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(False)
    for _ in range(3):
        logits.zero_()
        idx.fill_(-1)
        w.zero_()
        rb.storage.zero_()
        torch.cuda._sleep(4_000_000)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, want[0]) and torch.equal(w, want[1]) and torch.equal(rb.storage, want[2]) and int(err) == 0


# ---------------------------------------------------------------------------
# products
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


def make_rows(n_rows, n, seed):
    """FP8B rows whose blocks' scales differ, and their 64-bit values."""
    g = rnd(seed)
    v = torch.randn(n_rows, n, generator=g) * torch.exp(torch.randn(n_rows, 1, generator=g))
    size = torch.exp2(torch.randint(-2, 3, (n_rows, fp8b.blocks(n), 1), generator=g).float()).expand(-1, -1, 128)
    rows = fp8b.pack((v * size.reshape(n_rows, -1)[:, :n]).numpy())
    return torch.from_numpy(rows).cuda(), fp8b.values(rows, n)


def make_weights(E, parts, out, n, seed, scale):
    """Codes [E, parts, out, n], block scales, and their 64-bit values [E, parts * out, n]."""
    g = rnd(seed)
    size = torch.exp(0.5 * torch.randn(E, parts, fp8b.blocks(out), fp8b.blocks(n), generator=g)).numpy()
    w = torch.randn(E, parts, out, n, generator=g).numpy() * fp8b.spread_weights(size, out, n) * scale
    codes, s = fp8b.pack_weights(w.astype(np.float32))
    return (torch.from_numpy(codes).cuda(), torch.from_numpy(np.ascontiguousarray(s)).cuda(),
            fp8b.weight_values(codes, s).reshape(E, parts * out, n))


def check_product(L, R, T, E, n_in, n_out, out_dtype, swiglu, counts, bs=None, call_counts="given", stream=None):
    rows = E * R * T
    x, xv = make_rows(rows, n_in, 11 * E + n_in)
    w, ws, wv = make_weights(E, 1 + swiglu, n_out, n_in, 13 * E + n_out, n_in ** -0.5)
    at, v, err = ref.product(xv, wv, counts, T, swiglu)
    err = err * fp8b.product_error(n_in)
    unused = np.ones(rows, bool)
    unused[at] = False
    x[torch.from_numpy(unused)] = 0xFF  # rows that were not received: NaN codes and scales
    code = L.ROW_DTYPE_CODES
    rb = L.llmoe_row_bytes(n_out, code[out_dtype])
    y = torch.full((rows + 1, rb), 0xA5, dtype=torch.uint8, device="cuda")
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    if bs is None:
        bs = L.geometry(T, R, E, err=e)
    c = torch.from_numpy(counts).cuda() if call_counts == "given" else None
    torch.cuda.synchronize()
    L.llmoe_expert_product_fp8b(x, w, ws, y[:rows], c, n_in, n_out, code[out_dtype],
                                L.LLMOE_PRODUCT_SWIGLU if swiglu else 0, bs, stream)
    torch.cuda.synchronize()
    assert int(e) == 0
    y = y.cpu()
    assert (y[rows] == 0xA5).all() and (y[:rows][torch.from_numpy(unused)] == 0xA5).all()
    if not len(at):
        return
    got = y[:rows][torch.from_numpy(at)]
    if out_dtype == "fp8b":
        fp8b.check(got.numpy(), v, err)
    else:
        close(wide(got.contiguous().view(TORCH[out_dtype])), v, err, out_dtype)


# in, out: below one tile and one block, odd multiples, one tile, past an edge in either
PRODUCT_SIZES = [(16, 16), (48, 80), (128, 128), (144, 144), (256, 256), (272, 288), (640, 528), (1040, 48)]


@pytest.mark.parametrize("out_dtype,swiglu", [("bf16", False), ("fp16", False), ("fp32", False), ("bf16", True),
                                              ("fp16", True), ("fp32", True), ("fp8b", True)])
@pytest.mark.parametrize("n_in,n_out", PRODUCT_SIZES)
def test_product_types_and_sizes(L, n_in, n_out, out_dtype, swiglu):
    R, T, E = 2, 21, 4
    check_product(L, R, T, E, n_in, n_out, out_dtype, swiglu, some_counts(E, R, T, "ragged", n_in))


@pytest.mark.parametrize("n_out,out_dtype,swiglu", [(8, "bf16", False), (40, "fp16", False), (520, "bf16", False),
                                                    (4, "fp32", False), (132, "fp32", False), (264, "bf16", True),
                                                    (8, "fp32", True), (8, "bf16", True)])
def test_product_outputs_of_8_values(L, n_out, out_dtype, swiglu):
    check_product(L, 2, 33, 4, 176, n_out, out_dtype, swiglu, some_counts(4, 2, 33, "ragged", 3))


@pytest.mark.parametrize("kind", ["ragged", "full", "none", "one"])
@pytest.mark.parametrize("R,T,E", [(1, 1, 1), (1, 300, 3), (8, 5, 16), (40, 3, 40), (4, 130, 4), (3, 1, 96), (2, 64, 2)])
def test_product_geometries(L, R, T, E, kind):
    check_product(L, R, T, E, 160, 96, "bf16", False, some_counts(E, R, T, kind, R + T))
    check_product(L, R, T, E, 160, 96, "fp8b", True, some_counts(E, R, T, kind, R + T + 1))


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 63, 64, 65, 95, 97, 128, 160, 191, 193, 224, 225, 255, 256, 257, 481, 513])
def test_product_every_number_of_columns(L, rows):
    check_product(L, 1, rows, 1, 144, 144, "bf16", True, np.array([[rows]], np.int64))
    check_product(L, 1, rows, 1, 144, 272, "fp32", False, np.array([[rows]], np.int64))


def test_product_long_inner_dimension(L):
    check_product(L, 1, 40, 2, 4096, 64, "bf16", False, some_counts(2, 1, 40, "full", 0))
    check_product(L, 1, 300, 1, 7168, 256, "fp8b", True, some_counts(1, 1, 300, "full", 0))


@pytest.mark.parametrize("out_dtype,swiglu", [("bf16", False), ("fp8b", True)])
def test_product_many_tiles(L, out_dtype, swiglu):
    """More tiles than pairs of CTAs: every role goes around its rings."""
    check_product(L, 2, 300, 4, 784, 2320, out_dtype, swiglu, some_counts(4, 2, 300, "ragged", 5))


@pytest.mark.parametrize("out_dtype,swiglu", [("bf16", False), ("fp16", True), ("fp8b", True)])
@pytest.mark.parametrize("R,T", [(2, 64), (2, 68)])
def test_product_few_rows_and_many_steps(L, R, T, out_dtype, swiglu):
    """Room for 128 rows an expert, or for more: both kinds of ring, gone around in a tile."""
    c = some_counts(6, R, T, "ragged", R + T)
    c[2] = [T, 0]
    check_product(L, R, T, 6, 1168, 1040, out_dtype, swiglu, c)
    check_product(L, R, T, 6, 1168, 1040, out_dtype, swiglu, np.minimum(c, 3))


@pytest.mark.parametrize("T", [1, 40, 132])
def test_product_most_experts_of_few_rows(L, T):
    """Sums over 8192 experts take room of the ring."""
    c = some_counts(8192, 1, T, "ragged", T)
    c[np.random.RandomState(T).rand(8192, 1) < 0.9] = 0
    c[[0, 4095, 8191]] = T
    check_product(L, 1, T, 8192, 1168 if T == 1 else 16, 16, "bf16", False, c)


def test_product_on_another_stream(L):
    s = torch.cuda.Stream()
    check_product(L, 2, 17, 4, 128, 128, "bf16", True, some_counts(4, 2, 17, "ragged", 9), stream=s)


def test_product_is_reproducible_and_captures(L):
    """The same bits on every call, eager and replayed from a CUDA graph."""
    R, T, E, n_in, n_out = 2, 70, 6, 256, 320
    x, _ = make_rows(E * R * T, n_in, 1)
    w, ws, _ = make_weights(E, 2, n_out, n_in, 2, 0.1)
    c = torch.from_numpy(some_counts(E, R, T, "ragged", 4)).cuda()
    bs = L.geometry(T, R, E)
    rb = fp8b.row_bytes(n_out)
    ys = [torch.zeros(E * R * T, rb, dtype=torch.uint8, device="cuda") for _ in range(3)]

    def call(y):
        L.llmoe_expert_product_fp8b(x, w, ws, y, c, n_in, n_out, L.LLMOE_DTYPE_FP8B, L.LLMOE_PRODUCT_SWIGLU, bs)

    call(ys[0])
    call(ys[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ys[2])
    ys[2].fill_(0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("out_dtype", ["bf16", "fp8b"])
def test_product_nan_stays_in_its_row_and_block(L, out_dtype):
    R, T, E, n_in, n_out = 1, 40, 2, 256, 256
    counts = torch.tensor([[40], [7]], dtype=torch.int64, device="cuda")
    swiglu = out_dtype == "fp8b"
    x, _ = make_rows(E * R * T, n_in, 1)
    w, ws, _ = make_weights(E, 1 + swiglu, n_out, n_in, 2, 0.1)
    rb = L.llmoe_row_bytes(n_out, L.ROW_DTYPE_CODES[out_dtype])

    def run():
        y = torch.zeros(E * R * T, rb, dtype=torch.uint8, device="cuda")
        L.llmoe_expert_product_fp8b(x, w, ws, y, counts, n_in, n_out, L.ROW_DTYPE_CODES[out_dtype], int(swiglu),
                                    L.geometry(T, R, E))
        return y.cpu()

    clean = run()
    x[5, n_in:n_in + 4] = 255  # the NaN scale of one block of row 5
    x[6, 3] = 127  # a NaN code in row 6
    ws[1, 0, 1, 0] = float("inf")  # features 128.. of expert 1
    got = run()
    same = np.ones(E * T, bool)
    same[[5, 6]] = False
    same[T:T + 7] = False
    assert torch.equal(got[torch.from_numpy(same)], clean[torch.from_numpy(same)])
    if swiglu:
        q, s, _ = fp8b.split(got.numpy(), n_out)
        assert np.isnan(s[5:7]).all() and np.isnan(q[5:7]).all()
        assert np.isnan(s[T:T + 7, 1]).all()
        assert torch.equal(got[T:T + 7, :128], clean[T:T + 7, :128])
        assert torch.equal(got[T:T + 7, n_out:n_out + 4], clean[T:T + 7, n_out:n_out + 4])
    else:
        v, c = got.view(torch.bfloat16), clean.view(torch.bfloat16)
        assert v[5:7].isnan().all()
        assert torch.equal(v[T:T + 7, :128], c[T:T + 7, :128]) and not v[T:T + 7, 128:].isfinite().any()


@pytest.mark.parametrize("bad", [-3, 18])
def test_product_bad_count_is_reported_and_clamped(L, bad):
    R, T, E = 1, 17, 2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, xv = make_rows(E * R * T, 64, 1)
    w, ws, wv = make_weights(E, 1, 64, 64, 2, 1.0)
    y = torch.zeros(E * R * T + 1, 64, dtype=torch.bfloat16, device="cuda")
    bs = L.geometry(T, R, E, err=err)
    c = torch.tensor([[2], [bad]], dtype=torch.int64, device="cuda")
    L.llmoe_expert_product_fp8b(x, w, ws, y[:-1], c, 64, 64, 0, 0, bs)
    assert L.llmoe_get_error(bs) == L.LLMOE_DEV_SLOT_RANGE
    at, v, e = ref.product(xv, wv, np.array([[2], [min(max(bad, 0), T)]]), T, False)
    close(wide(y)[at], v, e * fp8b.product_error(64), "bf16")
    rest = np.ones(len(y), bool)
    rest[at] = False
    assert not wide(y)[rest].any()


@pytest.mark.parametrize("swiglu", [False, True])
def test_product_most_experts(L, swiglu):
    R, T, E = 1, 1, 8192
    c = (np.random.RandomState(3).rand(E, 1) < 0.3).astype(np.int64)
    check_product(L, R, T, E, 32, 32, "fp8b" if swiglu else "bf16", swiglu, c)


@pytest.mark.parametrize("n_in,n_out", [(8192, 64), (64, 4096)])
def test_product_offsets_past_32_bits(L, n_in, n_out):
    """x or y larger than 4 GiB, rows received at the very end of it."""
    R, T, E = 1, 80000, 8
    rows = E * R * T
    counts = np.array([[2], [0], [0], [5], [0], [0], [0], [T]], np.int64)
    used = np.concatenate([np.arange(2), np.arange(3 * T, 3 * T + 5), np.arange(rows - 3, rows)])
    x = torch.zeros(rows, fp8b.row_bytes(n_in), dtype=torch.uint8, device="cuda")
    xr, xv = make_rows(len(used), n_in, 5)
    x[torch.from_numpy(used).cuda()] = xr
    w, ws, wv = make_weights(E, 1, n_out, n_in, 6, n_in ** -0.5)
    y = torch.zeros(rows, n_out, dtype=torch.bfloat16, device="cuda")
    L.llmoe_expert_product_fp8b(x, w, ws, y, torch.from_numpy(counts).cuda(), n_in, n_out, 0, 0, L.geometry(T, R, E))
    got = wide(y[torch.from_numpy(used).cuda()])
    for i, r in enumerate(used):
        b = wv[r // T]
        close(got[i], b @ xv[i], (n_in + 80) * 2.0 ** -23 * (np.abs(b) @ np.abs(xv[i])), "bf16")
    assert not bool(y[2:3 * T].any()) and not bool(y[3 * T + 5:7 * T].any())
    del x, y
    torch.cuda.empty_cache()


def test_product_weights_past_32_bits(L):
    """Weights larger than 4 GiB: the last expert's last features."""
    R, T, E, n_in, n_out = 1, 3, 40, 7168, 16384  # 4.7 GB
    w = torch.zeros(E, 1, n_out, n_in, dtype=torch.uint8, device="cuda")
    ws = torch.ones(E, 1, n_out // 128, n_in // 128, device="cuda")
    last, s, wv = make_weights(1, 1, 200, n_in, 8, n_in ** -0.5)
    w[-1, 0, -200:] = last[0, 0]
    # the tail's two blocks: 72 features in the last but one, 128 in the last
    codes, sc = fp8b.pack_weights(np.concatenate([np.zeros((56, n_in), np.float32), wv[0].astype(np.float32)]))
    w[-1, 0, -256:] = torch.from_numpy(codes).cuda()
    ws[-1, 0, -2:] = torch.from_numpy(np.ascontiguousarray(sc)).cuda()
    x, xv = make_rows(E * R * T, n_in, 9)
    counts = torch.zeros(E, R, dtype=torch.int64)
    counts[-1, 0] = T
    y = torch.zeros(E * R * T, n_out, dtype=torch.bfloat16, device="cuda")
    L.llmoe_expert_product_fp8b(x, w, ws, y, counts.cuda(), n_in, n_out, 0, 0, L.geometry(T, R, E))
    b = fp8b.weight_values(codes, sc)
    for i in range(T):
        a = xv[(E - 1) * T + i]
        close(wide(y[(E - 1) * T + i])[-256:], b @ a, (n_in + 80) * 2.0 ** -23 * (np.abs(b) @ np.abs(a)), "bf16")
    assert not bool(y[:-T].any()) and not bool(y[-T:, :-256].any())
    del w, y
    torch.cuda.empty_cache()


def test_product_of_tensors_16_bytes_off(L):
    """Every pointer aligned as documented and no more."""
    R, T, E, n_in, n_out = 2, 11, 4, 160, 96
    counts = some_counts(E, R, T, "ragged", 8)
    x, xv = make_rows(E * R * T, n_in, 1)
    w, ws, wv = make_weights(E, 1, n_out, n_in, 2, 0.1)

    def shift(t, by):
        raw = t.reshape(-1).view(torch.uint8)
        return torch.cat([torch.zeros(by, dtype=torch.uint8, device="cuda"), raw])[by:]

    y = torch.zeros(16 + E * R * T * n_out * 2, dtype=torch.uint8, device="cuda")[16:]
    L.llmoe_expert_product_fp8b(shift(x, 16), shift(w, 16), shift(ws, 4).view(torch.float32), y,
                                torch.from_numpy(counts).cuda(), n_in, n_out, 0, 0, L.geometry(T, R, E))
    at, v, err = ref.product(xv, wv, counts, T, False)
    close(wide(y.view(torch.bfloat16).reshape(-1, n_out))[at], v, err * fp8b.product_error(n_in), "bf16")


def test_product_many_calls(L):
    """Calls with cold caches, warm ones and after other kernels: the same bits
    every time and no wait that expires."""
    R, T, E, K, n_in, n_out = 1, 128, 256, 8, 2048, 512
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bs = L.geometry(T, R, E, err=err)
    g = rnd(31)
    x = make_rows(E * R * T // 64, n_in, 1)[0].repeat(64, 1)
    w, ws, _ = make_weights(16, 2, n_out, n_in, 2, 0.05)
    w, ws = w.repeat(16, 1, 1, 1), ws.repeat(16, 1, 1, 1)
    flush = torch.empty(64 << 20, dtype=torch.float32, device="cuda")
    for _ in range(6):
        counts = torch.zeros(E, R, dtype=torch.int64)
        counts[torch.randperm(E, generator=g)[:K]] = 1
        c = counts.cuda()
        first = None
        for call in range(40):
            y = torch.zeros(E * R * T, fp8b.row_bytes(n_out), dtype=torch.uint8, device="cuda")
            if call % 4 == 1:
                flush.add_(1)
            L.llmoe_expert_product_fp8b(x, w, ws, y, c, n_in, n_out, L.LLMOE_DTYPE_FP8B, L.LLMOE_PRODUCT_SWIGLU, bs)
            first = y if first is None else first
            assert torch.equal(first, y)
        assert int(err) == 0
        assert int(first.any(1).sum()) == K


def test_products_on_two_streams_at_once(L):
    """Two calls in flight, each with every SM in its grid, one of them the MX8 product."""
    R, T, E, n = 2, 200, 8, 512
    c = torch.from_numpy(some_counts(E, R, T, "ragged", 6)).cuda()
    bs = L.geometry(T, R, E)
    x, _ = make_rows(E * R * T, n, 3)
    w, ws, _ = make_weights(E, 2, n, n, 4, 0.05)
    mx = torch.from_numpy(ref.pack_mx8(np.random.RandomState(1).randn(E * R * T, n))).cuda()
    mw = torch.from_numpy(ref.pack_mx8(np.random.RandomState(2).randn(E * n, n))).cuda()
    ys = [torch.zeros(E * R * T, fp8b.row_bytes(n), dtype=torch.uint8, device="cuda") for _ in range(2)]
    zs = [torch.zeros(E * R * T, n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s = [torch.cuda.Stream() for _ in range(2)]

    def pair(i, sa, sb):
        L.llmoe_expert_product_fp8b(x, w, ws, ys[i], c, n, n, L.LLMOE_DTYPE_FP8B, L.LLMOE_PRODUCT_SWIGLU, bs, sa)
        L.llmoe_expert_product(mx, mw, zs[i], c, n, n, L.LLMOE_DTYPE_MX8, 0, 0, bs, sb)

    torch.cuda.synchronize()
    pair(0, None, None)
    torch.cuda.synchronize()
    for _ in range(5):
        pair(1, *s)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(zs[0], zs[1]) and bool(ys[0].any())


def test_counts_from_the_rank_buffers(L):
    """FP8B rows through a dispatch, the product driven by its count words (counts NULL)."""
    R, T, E, K, n_in, n_out = 2, 9, 6, 2, 528, 64
    rb_in = fp8b.row_bytes(n_in)
    x, _ = make_rows(R * T, n_in, 3)
    w, ws, _ = make_weights(E, 1, n_out, n_in, 4, 0.05)
    idx = torch.rand(R, T, E, generator=rnd(1)).argsort(-1)[..., :K].contiguous()
    idx[0, 3, 1] = -1
    rb = L.RankBuffers(T, rb_in // 2, R, E, fill=0xA5)
    recv = torch.zeros(E * R * T, rb_in, dtype=torch.uint8, device="cuda")
    src = torch.zeros(E * R * T, dtype=torch.int32, device="cuda")
    for s in (0, 1):
        bs = rb.buf_set(s, K)
        L.llmoe_clean(bs)
        L.llmoe_dispatch_unpack(x.view(torch.bfloat16), idx.cuda(), recv.view(torch.bfloat16), src, bs)
        counts = torch.empty(E, R, dtype=torch.int64, device="cuda")
        slot = torch.empty(R, T, K, dtype=torch.int32, device="cuda")
        L.llmoe_route(idx.cuda(), slot, counts, bs)
        ya, yb = (torch.zeros(E * R * T, n_out, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        L.llmoe_expert_product_fp8b(recv, w, ws, ya, None, n_in, n_out, 0, 0, bs)
        L.llmoe_expert_product_fp8b(recv, w, ws, yb, counts, n_in, n_out, 0, 0, L.geometry(T, R, E))
        assert torch.equal(ya, yb) and bool(ya.any())


# ---------------------------------------------------------------------------
# one MoE block
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("coded,dtype", [(False, "bf16"), (True, "bf16"), (False, "fp16")])
def test_moe_block(L, coded, dtype):
    """The whole block against its definition, given its own logits and rows."""
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock, pack_fp8b_weights

    R, T, n, H, I, E, K, G, kept = 2, 24, 19, 528, 176, 16, 3, 4, 2
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
    gu_codes, gu_s = fp8b.pack_weights(gate_up.float().numpy().reshape(E, 2, I, H))
    dn_codes, dn_s = fp8b.pack_weights(down.float().numpy())
    gu, dn = fp8b.weight_values(gu_codes, gu_s).reshape(E, 2 * I, H), fp8b.weight_values(dn_codes, dn_s)
    kw = dict(router_bias=bias.cuda(), dtype=dtype, rows="fp8b", scale=2.0, err=err, num_groups=G, kept_groups=kept,
              group_top2=True)
    if coded:
        a, b = pack_fp8b_weights(gate_up.cuda().reshape(E, 2, I, H))
        c, d = pack_fp8b_weights(down.cuda())
        m = MoEBlock(T, R, K, norm_w.cuda(), router_w.cuda(), a.reshape(E, 2 * I, H).view(torch.float8_e4m3fn), c,
                     gate_up_scale=b, down_scale=d, **kw)
    else:
        m = MoEBlock(T, R, K, norm_w.cuda(), router_w.cuda(), gate_up.cuda(), down.cuda(), **kw)
    residual, out = res.cuda(), torch.full((R, n, H), float("nan"), dtype=t, device="cuda")
    m.forward(x.cuda(), residual, out, active.cuda())
    first = out.clone()
    h = (x.float() + res.float()).to(t)
    assert torch.equal(residual.cpu(), h)
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
    fp8b.check(m.rows.cpu().numpy()[:tokens], v, np.abs(v) * NORM_ERR)
    logits = m.logits[:tokens].cpu().numpy()
    idx, topk_w = m.topk_idx[:tokens].cpu().numpy(), wide(m.topk_w)[:tokens]
    seen = 0
    for r in range(tokens):
        want, ww, gap = fp8b.group_router(logits[r:r + 1], bias.numpy(), active.reshape(-1)[r:r + 1].numpy(), K, G, kept,
                                          True, "sigmoid", True, 2.0)
        if gap > 4e-6:
            seen += 1
            assert np.array_equal(idx[r], want[0]) and np.allclose(topk_w[r], ww[0], rtol=64 * 2.0 ** -23, atol=0)
    assert seen > tokens // 2
    xe = fp8b.values(m.rows.cpu().numpy()[:tokens], H)
    got = wide(first).reshape(tokens, H)
    for i in range(tokens):
        total, tol = np.zeros(H), np.zeros(H)
        for k in range(K):
            e = idx[i, k]
            if e < 0:
                continue
            _, hv, he = ref.product(xe[i:i + 1], gu[e:e + 1], np.array([[1]]), 1, True)
            hv, he = hv[0], he[0] * fp8b.product_error(H)
            # h's rounding to e4m3: half a step of its block's largest value bounds it
            he = he + 2.0 ** -4 * fp8b.spread(fp8b.block_max(np.abs(hv) + he), I) + TINY[dtype]
            y = dn[e] @ hv
            ye = np.abs(dn[e]) @ he + (I + 4) * 2.0 ** -23 * (np.abs(dn[e]) @ np.abs(hv))
            ye += (np.abs(y) + ye) * HALF_ULP[dtype] + TINY[dtype]
            total += topk_w[i, k] * y
            tol += topk_w[i, k] * ye
        tol += (np.abs(total) + tol) * (HALF_ULP[dtype] + K * 2.0 ** -23) + TINY[dtype]
        assert (np.abs(got[i] - total) <= tol).all(), i


def test_moe_block_queued(L):
    """A block's calls all queued while the device is still busy, over buffers
    that held something else: the bits of a call on an idle device."""
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    R, T, n, H, I, E, K = 4, 64, 37, 1536, 768, 32, 4
    g = rnd(91)
    new = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(torch.bfloat16).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = MoEBlock(T, R, K, torch.ones(H, dtype=torch.bfloat16, device="cuda"), new(E, H), new(E, 2 * I, H), new(E, H, I),
                 None, "bf16", "fp8b", err=err, num_groups=8, kept_groups=4, group_top2=True)
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
        m.h.zero_()
        torch.cuda.synchronize()
        if busy:
            torch.cuda._sleep(8_000_000)
        m.forward(x, res, out)
        torch.cuda.synchronize()
        assert int(err) == 0
        outs.append(out.clone())
    assert torch.isfinite(outs[0]).all() and (outs[0] != 0).any()
    assert torch.equal(outs[1], outs[0]) and torch.equal(outs[2], outs[0])
