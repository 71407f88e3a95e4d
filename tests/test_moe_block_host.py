"""Refusals of MoEBlock: every call below raises ValueError before anything is
launched or written, so it runs on tensors of the CPU, without a GPU."""
import pytest
import torch

T, R, n, H, I, E, K = 6, 2, 4, 64, 32, 4, 2


@pytest.fixture(scope="module")
def Block():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    return MoEBlock


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def arguments(**kw):
    a = dict(num_max_tokens=T, num_ranks=R, num_topk=K, norm_weight=z(H), router_weight=z(E, H), gate_up=z(E, 2 * I, H),
             down=z(E, H, I))
    a.update(kw)
    return a


@pytest.mark.parametrize("what,kw", [
    ("norm_weight", dict(norm_weight=z(H + 8))), ("norm_weight", dict(norm_weight=z(1, H))),
    ("norm_weight", dict(norm_weight=z(H, dtype=torch.float32))),
    ("router_weight", dict(router_weight=z(E, H, dtype=torch.float16))),
    ("router_weight", dict(router_weight=z(E, H, 1))),
    ("router_weight", dict(router_weight=z(H, E).T)),
    ("gate_up", dict(gate_up=z(E, 2 * I, H + 8))), ("gate_up", dict(gate_up=z(E, I, H))),
    ("gate_up", dict(gate_up=z(E - 1, 2 * I, H))), ("gate_up", dict(gate_up=z(E, 2 * I, H, dtype=torch.float32))),
    ("gate_up", dict(gate_up=z(E, H, 2 * I).transpose(1, 2))),
    ("gate_up", dict(down=z(E, I, H))), ("down", dict(down=z(E, H, I, dtype=torch.float32))), ("down", dict(down=z(H, I))),
    ("down", dict(down=z(E + 2, H, I))),
    ("router_bias", dict(router_bias=z(E))), ("router_bias", dict(router_bias=z(E + 1, dtype=torch.float32))),
    ("dtype", dict(dtype="fp32")), ("rows", dict(rows="fp8")),
    ("num_topk", dict(num_topk=0)), ("num_topk", dict(num_topk=E + 1)),
    ("num_max_tokens", dict(num_max_tokens=0)), ("num_ranks", dict(num_ranks=0)), ("num_ranks", dict(num_ranks=3)),
    ("hidden", dict(norm_weight=z(60), router_weight=z(E, 60), gate_up=z(E, 2 * I, 60), down=z(E, 60, I))),
    ("hidden", dict(gate_up=z(E, 2 * 12, H), down=z(E, H, 12))),
    ("hidden", dict(rows="mx8", gate_up=z(E, 2 * 40, H), down=z(E, H, 40))),
    ("device", dict(down=torch.zeros(E, H, I, dtype=torch.bfloat16, device="meta"))),
])
def test_weights(Block, what, kw):
    with pytest.raises(ValueError, match=rf"\b{what}\b"):
        Block(**arguments(**kw))


def inputs(**kw):
    a = dict(x=z(R, n, H), residual=z(R, n, H), out=z(R, n, H), active=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("what,kw", [
    ("x", dict(x=z(R, n, H + 8))), ("x", dict(x=z(R, n, H // 2))), ("x", dict(x=z(R * n, H))),
    ("x", dict(x=z(R, n, H, dtype=torch.float32))), ("x", dict(x=z(R, n, H, dtype=torch.float16))),
    ("x", dict(x=z(R, H, n).transpose(1, 2))), ("ranks", dict(x=z(R + 1, n, H))), ("tokens", dict(x=z(R, T + 1, H))),
    ("residual", dict(residual=z(R, n - 1, H))), ("residual", dict(residual=z(1, n, H))),
    ("residual", dict(residual=z(R, n, H, dtype=torch.float32))), ("residual", dict(residual=z(n, R, H).transpose(0, 1))),
    ("out", dict(out=z(R, n, H // 2))), ("out", dict(out=z(R, n - 1, H))), ("out", dict(out=z(R, n, H, dtype=torch.float16))),
    ("out", dict(out=z(R, n, H)[:, :, ::2])),
    ("active", dict(active=torch.ones(R, n - 1, dtype=torch.uint8))), ("active", dict(active=torch.ones(R * n, dtype=torch.uint8))),
    ("active", dict(active=torch.ones(R, n, dtype=torch.int64))),
    ("active", dict(active=torch.ones(n, R, dtype=torch.uint8).T)),
    ("device", dict(residual=torch.zeros(R, n, H, dtype=torch.bfloat16, device="meta"))),
])
def test_activations(Block, what, kw):
    m = Block(**arguments())
    with pytest.raises(ValueError, match=rf"\b{what}\b"):
        m.forward(**inputs(**kw))


def test_out_over_the_residual(Block):
    """Both are results: one memory cannot hold them."""
    m = Block(**arguments())
    r = z(R, n, H)
    with pytest.raises(ValueError, match="overlap"):
        m.forward(z(R, n, H), r, r)
    flat = z(2 * R * n * H)
    with pytest.raises(ValueError, match="overlap"):
        m.forward(z(R, n, H), flat[:R * n * H].view(R, n, H), flat[H:H + R * n * H].view(R, n, H))


@pytest.mark.parametrize("name", ["x", "residual", "out"])
def test_alignment(Block, name):
    m = Block(**arguments())
    flat = z(R * n * H + 8)
    at = next(i for i in range(8) if (flat.data_ptr() + 2 * i) % 16 == 2)
    with pytest.raises(ValueError, match="aligned"):
        m.forward(**inputs(**{name: flat[at:at + R * n * H].view(R, n, H)}))


def test_experts_in_fours(Block):
    """The router's logits are fp32 rows of whole 16 bytes."""
    m = Block(**arguments(router_weight=z(2, H), gate_up=z(2, 2 * I, H), down=z(2, H, I)))
    with pytest.raises(ValueError, match="multiple of 4"):
        m.forward(**inputs())
