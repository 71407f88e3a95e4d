"""GPU test of the weights that MoEBlock's router gives, renormalised and not: against
the router's definition on the block's own logits, and the output that they scale.
Weights: exponential, sum over E and division, a rounding each per term (as in
test_gpu_scaled.py).  Outputs: with one expert a token the output is its row times
the weight, so two blocks' outputs are in the ratio of their weights, to bf16's
rounding of either (2^-8 each) and of the product in fp32."""
import numpy as np
import pytest
import torch

import fp8b_reference as fp8b

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return llmoe


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
@pytest.mark.parametrize("K", [1, 3])
def test_weights(L, K, groups, kept, scoring):
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    R, T, H, I, E = 2, 13, 256, 128, 16
    g = torch.Generator().manual_seed(K + groups)
    new = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).bfloat16().cuda()
    norm_w, router_w, gate_up, down = torch.ones(H, dtype=torch.bfloat16, device="cuda"), new(E, H), new(E, 2 * I, H), new(E, H, I)
    x, res = H ** 0.5 * new(R, T, H), new(R, T, H)
    code = L.LLMOE_SCORE_SIGMOID if scoring == "sigmoid" else L.LLMOE_SCORE_SOFTMAX
    outs, weights = [], []
    for renorm in (True, False):
        m = MoEBlock(T, R, K, norm_w, router_w, gate_up, down, None, "bf16", "fp8b", scale=1.5, scoring=code,
                     num_groups=groups, kept_groups=kept, renorm=renorm)
        out = torch.empty_like(x)
        m.forward(x, res.clone(), out)
        logits, idx, w = m.logits.cpu().numpy(), m.topk_idx.cpu().numpy(), m.topk_w.cpu().double().numpy()
        seen = 0
        for r in range(R * T):
            want, ww, gap = fp8b.group_router(logits[r:r + 1], None, None, K, groups, kept, False, scoring, renorm, 1.5)
            if gap < 1e-5:
                continue
            seen += 1
            assert np.array_equal(idx[r], want[0])
            assert (np.abs(w[r] - ww[0]) <= ww[0] * (E / 32 + K + 32) * 2.0 ** -23).all()
        assert seen > R * T // 2
        outs.append(out.double().cpu().numpy().reshape(R * T, H))
        weights.append(w)
    if K == 1 or scoring == "softmax":  # scores of a sum below 1
        assert (weights[0].sum(1) > weights[1].sum(1)).all()
    if K == 1:
        a, b = (o / w for o, w in zip(outs, weights))
        assert (np.abs(a - b) <= (np.abs(a) + np.abs(b)) * (2.0 ** -8 + 2.0 ** -22)).all()
    # a block that does not say is renormalised
    m = MoEBlock(T, R, K, norm_w, router_w, gate_up, down, None, "bf16", "fp8b", scale=1.5, scoring=code,
                 num_groups=groups, kept_groups=kept)
    out = torch.empty_like(x)
    m.forward(x, res.clone(), out)
    assert np.array_equal(out.double().cpu().numpy().reshape(R * T, H), outs[0])
