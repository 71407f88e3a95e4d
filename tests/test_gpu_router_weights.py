"""GPU tests of the router's weights where masks and extreme logits decide them
(include/llmoe_block.h): which experts a softmax is over, and weights whose
scores are too small for fp32 or whose sum is.

The reference is written from the header in 64 bits: a softmax over the experts
that can be chosen, and with LLMOE_ROUTER_RENORM the softmax over the chosen
ones, which is what scale * score / sum is.

Tolerance of a weight: an exponential of a difference d (2 ulp, and half an ulp
of d in its argument, d below 128: 2^-18 relative), a sum of at most E of them in
E / 32 + 5 steps and K + 5 more, a division and two products.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# experts: one to a lane, several, more than a warp holds in registers, and not a multiple of four
EXPERTS = [8, 40, 256, 255, 600, 2050]


@pytest.fixture(scope="module")
def L():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return llmoe


def softmax_of(v):
    """Of 64-bit logits; those of +infinity share the weight."""
    if (v == np.inf).any():
        e = (v == np.inf).astype(float)
    else:
        e = np.exp(v - v.max())
    return e / e.sum()


def softmax_router(logits, bias, K, renorm, scale):
    """idx and w of each row, from the header."""
    rows, E = logits.shape
    idx, w = np.full((rows, K), -1, np.int64), np.zeros((rows, K))
    for r in range(rows):
        l = logits[r].astype(np.float64)
        with np.errstate(invalid="ignore"):
            key = l + (0 if bias is None else bias.astype(np.float64))
        can = [e for e in range(E) if l[e] > -np.inf and key[e] > -np.inf]
        if not can:
            continue
        chosen = sorted(can, key=lambda e: (-key[e], e))[:K]
        idx[r, :len(chosen)] = chosen
        if renorm:
            w[r, :len(chosen)] = scale * softmax_of(l[chosen])
        else:
            score = dict(zip(can, softmax_of(l[can])))
            w[r, :len(chosen)] = [scale * score[e] for e in chosen]
    return idx, w


def run(L, logits, bias, K, scoring, renorm, scale):
    rows, E = logits.shape
    idx = torch.full((rows, K), -7, dtype=torch.int64, device="cuda")
    w = torch.full((rows, K), NAN, device="cuda")
    L.llmoe_topk_router(logits.cuda(), None if bias is None else bias.cuda(), None, idx, w, rows, E, K,
                        L.LLMOE_DTYPE_FP32, scoring, L.LLMOE_ROUTER_RENORM if renorm else 0, scale)
    return idx.cpu().numpy(), w.cpu().double().numpy()


def check(L, logits, bias, K, renorm, scale=2.5):
    gi, gw = run(L, logits, bias, K, L.LLMOE_SCORE_SOFTMAX, renorm, scale)
    idx, w = softmax_router(logits.numpy(), None if bias is None else bias.numpy(), K, renorm, scale)
    assert np.array_equal(gi, idx)
    E = logits.shape[1]
    tol = w * (2.0 ** -18 + (E / 32 + K + 24) * 2.0 ** -23) + scale * 2.0 ** -126  # a subnormal weight may be off by all of it
    bad = ~(np.abs(gw - w) <= tol)
    assert not bad.any(), (gw[bad][:4], w[bad][:4])


def eighths(rows, E, seed):
    """Logits on a grid of 1/8, exact in fp32 with the biases below."""
    return torch.randint(-24, 25, (rows, E), generator=torch.Generator().manual_seed(seed)).float() / 8


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", EXPERTS)
def test_softmax_leaves_out_experts_that_the_bias_masks(L, E, renorm):
    """Masked by a bias of -infinity or NaN, their logits far above the rest,
    +infinity among them: the others' weights are those of a softmax without them."""
    K = 3
    logits = eighths(6, E, E)
    bias = torch.zeros(E)
    masked = [1, 5, E - 2]
    bias[masked[0]], bias[masked[1]], bias[masked[2]] = -INF, NAN, -INF
    logits[0, masked[0]] = 20.0
    logits[1, masked[2]] = 70.0  # the others' share is 1e-30
    logits[2, masked] = 100.0  # ... and not in fp32
    logits[3, masked[0]] = INF
    logits[4, masked[1]] = INF
    logits[5] = torch.finfo(torch.float32).min  # the type's lowest everywhere but there
    logits[5, masked] = 3.0
    check(L, logits, bias, K, renorm)


@pytest.mark.parametrize("E", EXPERTS)
def test_softmax_rows_without_a_choice(L, E):
    logits = eighths(3, E, 2 * E)
    bias = torch.full((E,), -INF)
    for renorm in (False, True):
        gi, gw = run(L, logits, bias, 2, L.LLMOE_SCORE_SOFTMAX, renorm, 1.0)
        assert (gi == -1).all() and (gw == 0).all()


@pytest.mark.parametrize("lead", [60.0, 95.0, 120.0, 1e4])
@pytest.mark.parametrize("E", EXPERTS)
def test_renormalised_softmax_below_a_leading_expert(L, E, lead):
    """An expert whose logit leads by far but whose finite bias keeps it from
    being chosen: the chosen scores are too small for fp32, their shares are not."""
    logits = eighths(4, E, 3 * E)
    bias = torch.zeros(E)
    bias[2] = -1e6
    logits[:, 2] = lead
    check(L, logits, bias, 3, True)
    check(L, logits, None, 3, True)  # and chosen


@pytest.mark.parametrize("K", [1, 2, 4])
@pytest.mark.parametrize("E", EXPERTS)
def test_renormalised_sigmoid_of_least_scores(L, E, K):
    """Equal scores of about 5e-39 (subnormal): every weight is scale / K
    exactly, where scale / sum is above fp32's largest value."""
    logits = torch.full((5, E), -88.0)
    gi, gw = run(L, logits, None, K, L.LLMOE_SCORE_SIGMOID, True, 2.5)
    assert (gi == np.arange(K)).all()
    assert (gw == 2.5 / K).all()
    # a sum of zero gives zeros
    gi, gw = run(L, torch.full((5, E), -200.0), None, K, L.LLMOE_SCORE_SIGMOID, True, 2.5)
    assert (gi == np.arange(K)).all() and (gw == 0).all()


def test_inputs_and_outputs_side_by_side(L):
    """One allocation holds logits, bias, active, topk_idx and topk_w, each right
    behind the one before: no overlap, so no refusal."""
    rows, E, K = 8, 40, 3
    sizes = [rows * E * 4, E * 4, rows, rows * K * 8, rows * K * 4]
    flat = torch.zeros(sum(sizes), dtype=torch.uint8, device="cuda")
    logits, bias, active, idx, w = flat.split(sizes)
    want = eighths(rows, E, 5)
    logits.view(torch.float32).copy_(want.reshape(-1).cuda())
    active.fill_(1)
    L.llmoe_topk_router(logits.view(torch.float32), bias.view(torch.float32), active, idx.view(torch.int64),
                        w.view(torch.float32), rows, E, K, L.LLMOE_DTYPE_FP32, L.LLMOE_SCORE_SOFTMAX, 0, 1.0)
    ri, _ = softmax_router(want.numpy(), None, K, False, 1.0)
    assert np.array_equal(idx.view(torch.int64).cpu().numpy().reshape(rows, K), ri)
