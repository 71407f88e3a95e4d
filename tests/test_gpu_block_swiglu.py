"""GPU test of SwiGLU's arithmetic where the output type shows it: fp32 outputs
of the expert products (include/llmoe_block.h).

One input value is 1 and the others are 0, so that the gate's sum is a weight
and the up's is 1, both exactly; the output is silu of the weight.  Tolerance:
an exponential within 2 ulp, a sum, a division and a product rounded to nearest:
3.5 ulp of 2^-23 at most, 4 taken.
"""
import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300 import llmoe

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return llmoe


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "mx8"])
def test_silu_in_fp32(L, dtype):
    n_in, n_out, T = 64, 1024, 5
    # every eighth from -80 to 48, both ends included
    gate = torch.linspace(-80, 48, n_out + 1)[:n_out].double()
    if dtype != "mx8":
        gate = gate.to({"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]).double()
    w = torch.zeros(2 * n_out, n_in, dtype=torch.float64)
    w[:n_out, 7] = gate
    w[n_out:, 7] = 1
    x = torch.zeros(T, n_in, dtype=torch.float64)
    x[:, 7] = 1
    if dtype == "mx8":
        w, x = ref.pack_mx8(w.numpy()), ref.pack_mx8(x.numpy())
        gate = ref.mx8_values(w, n_in)[:n_out, 7]
        w, x = torch.from_numpy(w).cuda(), torch.from_numpy(x).cuda()
    else:
        t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        gate, w, x = gate.numpy(), w.to(t).cuda(), x.to(t).cuda()
    y = torch.full((T, n_out), float("nan"), device="cuda")
    counts = torch.tensor([[T]], dtype=torch.int64, device="cuda")
    L.llmoe_expert_product(x, w, y, counts, n_in, n_out, L.ROW_DTYPE_CODES[dtype], L.LLMOE_DTYPE_FP32,
                           L.LLMOE_PRODUCT_SWIGLU, L.geometry(T, 1, 1))
    want = gate / (1 + np.exp(-gate))
    got = y.cpu().double().numpy()
    off = np.abs(got - want) / np.maximum(np.abs(want), 2.0 ** -126)
    assert (off <= 4 * 2.0 ** -23).all(), (off.max() / 2.0 ** -23, gate[off.max(0).argmax()])
