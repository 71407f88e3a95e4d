"""MoEBlock refuses what its calls would refuse, when it is made: a call that
is refused behind the norm would leave the residual changed and no output."""
import pytest
import torch

T, R, H, I, E, K = 6, 2, 64, 48, 8, 2
bf16, u8, f32 = torch.bfloat16, torch.uint8, torch.float32


@pytest.fixture(scope="module")
def Block():
    from combine_routing_count_prefix_gb300 import build

    build.build()
    from combine_routing_count_prefix_gb300.moe_block import MoEBlock

    return MoEBlock


def off(*shape, dtype=bf16, by=8):
    """Zeros `by` bytes behind a 16-byte boundary, as a tensor inside a larger file may lie."""
    n = torch.Size(shape).numel() * dtype.itemsize
    raw = torch.zeros(n + 32, dtype=u8)
    at = next(i for i in range(16) if (raw.data_ptr() + i) % 16 == by)
    return raw[at:at + n].view(dtype).view(shape)


def arguments(rows, **kw):
    z = lambda *s, dtype=bf16: torch.zeros(*s, dtype=dtype)
    a = dict(num_max_tokens=T, num_ranks=R, num_topk=K, norm_weight=z(H), router_weight=z(E, H), gate_up=z(E, 2 * I, H),
             down=z(E, H, I), rows=rows)
    if rows == "fp8b":
        a.update(gate_up=z(E, 2 * I, H, dtype=u8), down=z(E, H, I, dtype=u8), gate_up_scale=z(E, 2, 1, 1, dtype=f32),
                 down_scale=z(E, 1, 1, dtype=f32))
    a.update(kw)
    return a


@pytest.mark.parametrize("rows", ["same", "fp8b"])
@pytest.mark.parametrize("name,shape", [("norm_weight", (H,)), ("router_weight", (E, H)), ("gate_up", (E, 2 * I, H)),
                                        ("down", (E, H, I))])
@pytest.mark.parametrize("by", [2, 8])
def test_weights_off_16_bytes(Block, rows, name, shape, by):
    coded = rows == "fp8b" and name in ("gate_up", "down")
    with pytest.raises(ValueError, match=rf"\b{name}\b.*aligned"):
        Block(**arguments(rows, **{name: off(*shape, dtype=u8 if coded else bf16, by=by)}))


@pytest.mark.parametrize("rows", ["same", "fp8b"])
def test_weights_on_16_bytes(Block, rows):
    Block(**arguments(rows, norm_weight=off(H, by=0)))


@pytest.mark.parametrize("scoring", [-1, 2, None])
def test_scoring(Block, scoring):
    with pytest.raises(ValueError, match="scoring"):
        Block(**arguments("same", scoring=scoring))
