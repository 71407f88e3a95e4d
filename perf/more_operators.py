"""Cases of the block-scaled MoE operators: what is timed and compared, and the operators' plain forms.

The operators are a MoE block's in the 8-bit form with a fp32 scale for each 128 values, and its
router with groups:

- ``router``: top-k experts of the groups that score best, with their weights;
- ``rows``: residual addition and RMS norm to FP8B rows, or FP8B rows of values as they are;
- ``pack``: weights as e4m3 codes with a fp32 scale for each 128 x 128 block;
- ``product``: matrix products grouped by expert of FP8B rows with such weights, optionally gate / up
  with SwiGLU, to 16 bits or to FP8B rows again.

Where ``own`` is false ``run`` computes them from elementary torch operations in 32 bits; where it is
true it makes the library's calls.

An FP8B row of n values is n e4m3 codes, then one fp32 scale for each 128 values (the last block may be
short), then zeros up to a multiple of 16 bytes.  A scale is its block's largest magnitude / 448, at
least 2^-126.

Received rows lie at (e * R + src) * T + slot, slot < counts[e][src]: the row order of the framework's
recv_x.  The other rows of an output keep what they held (zeros here).
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_B = 128  # values with one scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # routing one token: 256 experts in 8 groups, of which 4 are kept
        {"name": "router-one-token", "op": "router", "rows": 1, "experts": 256, "topk": 8, "groups": 8, "kept": 4,
         "dtype": "fp32", "scoring": "sigmoid", "top2": True, "bias": True, "renorm": True, "idle": 0.0},
        # the large batch, 8 ranks x 1024 tokens, a tenth of them padding
        {"name": "router-large", "op": "router", "rows": 8192, "experts": 256, "topk": 8, "groups": 8, "kept": 4,
         "dtype": "fp32", "scoring": "sigmoid", "top2": True, "bias": True, "renorm": True, "idle": 0.1},
        # softmax over 160 experts in groups of 20, by each group's best, 16-bit logits
        {"name": "router-softmax-160", "op": "router", "rows": 4096, "experts": 160, "topk": 6, "groups": 8, "kept": 3,
         "dtype": "bf16", "scoring": "softmax", "top2": False, "bias": False, "renorm": False, "idle": 0.0},
        # one token through the block's norm: a single sequence being decoded
        {"name": "rows-norm-one-token", "op": "rows", "rows": 1, "hidden": 7168, "dtype": "bf16", "norm": True,
         "residual": True},
        # the large batch's norm, written as the 8-bit rows that are dispatched
        {"name": "rows-norm-large", "op": "rows", "rows": 8192, "hidden": 7168, "dtype": "bf16", "norm": True,
         "residual": True},
        # one matrix of a ragged size: 2000 x 1040 fp32 values, short blocks at both edges
        {"name": "pack-one-ragged", "op": "pack", "matrices": 1, "rows": 2000, "cols": 1040, "dtype": "fp32"},
        # gate and up of 16 experts, as they are laid out when a model is loaded
        {"name": "pack-gate-up", "op": "pack", "matrices": 32, "rows": 2048, "cols": 7168, "dtype": "bf16"},
        # one token of one rank: eight experts with one row each, the weights read once
        {"name": "product-one-token", "op": "product", "out_type": "bf16", "R": 1, "T": 128, "tokens": 1, "E": 256,
         "K": 8, "in": 7168, "out": 2048, "swiglu": True, "zipf": 0.0, "mask": 0.0},
        # decode micro-batch, gate and up with SwiGLU to rows for the next product: about 32 rows for each of 256 experts
        {"name": "product-decode-gate-up", "op": "product", "out_type": "fp8b", "R": 8, "T": 128, "tokens": 128,
         "E": 256, "K": 8, "in": 7168, "out": 2048, "swiglu": True, "zipf": 0.0, "mask": 0.0},
        # skewed routing (Zipf 1.2, a tenth masked) and sizes that end inside a block and a tile
        {"name": "product-skewed-ragged", "op": "product", "out_type": "fp16", "R": 8, "T": 100, "tokens": 100, "E": 64,
         "K": 6, "in": 2000, "out": 4104, "swiglu": False, "zipf": 1.2, "mask": 0.1},
        # few experts, a thousand rows each: bound by the tensor cores
        {"name": "product-dense-gate-up", "op": "product", "out_type": "fp8b", "R": 8, "T": 256, "tokens": 256, "E": 16,
         "K": 8, "in": 7168, "out": 2048, "swiglu": True, "zipf": 0.0, "mask": 0.0},
        # their down projection: a short sum, so that the tiles' ends count
        {"name": "product-dense-down", "op": "product", "out_type": "bf16", "R": 8, "T": 256, "tokens": 256, "E": 16,
         "K": 8, "in": 2048, "out": 7168, "swiglu": False, "zipf": 0.0, "mask": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "rows", "pack", "product", "product", "product"])
    if op == "router":
        groups = rng.choice([2, 4, 8, 8, 16])
        experts = groups * _log(rng, 2, 512 // groups)
        kept = rng.randint(1, groups)
        scoring = rng.choice(["sigmoid", "sigmoid", "softmax"])
        return {"op": "router", "rows": min(_log(rng, 1, 8192), 8192 * 256 // experts), "experts": experts,
                "topk": rng.randint(1, min(8, experts // groups * kept)), "groups": groups, "kept": kept,
                "dtype": rng.choice(["fp32", "fp32", "bf16"]), "scoring": scoring,
                "top2": scoring == "sigmoid" and rng.random() < 0.75, "bias": rng.random() < 0.5,
                "renorm": rng.random() < 0.75, "idle": rng.choice([0.0, 0.1])}
    if op == "rows":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        hidden = 16 * _log(rng, 4, 512)
        norm = rng.random() < 0.75
        return {"op": "rows", "rows": min(_log(rng, 1, 8192), 8192 * 7168 * 2 // (hidden * _BYTES[dtype])),
                "hidden": hidden, "dtype": dtype, "norm": norm, "residual": norm and rng.random() < 0.75}
    if op == "pack":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        rows, cols = _log(rng, 32, 8192), 16 * _log(rng, 4, 512)
        most = 32 * 2048 * 7168 * 2 // (rows * cols * _BYTES[dtype])
        return {"op": "pack", "matrices": max(1, min(_log(rng, 1, 64), most)), "rows": rows, "cols": cols,
                "dtype": dtype}
    R = rng.choice([1, 2, 4, 8])
    E = R * _log(rng, 1, 256 // R)
    tokens = _log(rng, 1, 256)
    swiglu = rng.random() < 0.5
    n_in = 16 * _log(rng, 16, 7168 // 16)
    n_out = 16 * _log(rng, 16, 2048 // 16) if swiglu else 8 * _log(rng, 32, 7168 // 8)
    K = min(E, rng.choice([1, 2, 4, 6, 8]))
    # no dearer than the listed cases: the decode case's weights, the dense case's operations
    while (E * (2 if swiglu else 1) * n_out * n_in > 7_500_000_000
           or R * tokens * K * (2 if swiglu else 1) * n_out * n_in > 8 * 256 * 8 * 4096 * 7168):
        n_out = max(16, n_out // 32 * 16)
    return {"op": "product", "out_type": rng.choice(["fp8b", "bf16"] if swiglu else ["bf16", "fp16"]), "R": R,
            "T": tokens + rng.randint(0, 16), "tokens": tokens, "E": E, "K": K, "in": n_in, "out": n_out,
            "swiglu": swiglu, "zipf": rng.choice([0.0, 0.0, 1.2]), "mask": rng.choice([0.0, 0.1])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _blocks(n):
    return -(-n // _B)


def _row_bytes(n, dtype):
    return n + -(-4 * _blocks(n) // 16) * 16 if dtype == "fp8b" else n * _BYTES[dtype]


def _codes(v, scale):
    """32-bit values over the scales they lie behind, as e4m3."""
    return (v * (1 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn)


def _pack_rows(v):
    """32-bit values [rows, n] as FP8B rows, uint8 [rows, row bytes]."""
    rows, n = v.shape
    p = torch.nn.functional.pad(v, (0, _blocks(n) * _B - n)).reshape(rows, -1, _B)
    scale = (p.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    out = torch.zeros(rows, _row_bytes(n, "fp8b"), dtype=torch.uint8, device=v.device)
    out[:, :n] = _codes(p, scale[..., None]).reshape(rows, -1)[:, :n].view(torch.uint8)
    out[:, n:n + 4 * _blocks(n)] = scale.contiguous().view(torch.uint8)
    return out


def _pack_weights(w):
    """32-bit values [matrices, rows, cols] as e4m3 codes and the scales of their 128 x 128 blocks."""
    m, rows, cols = w.shape
    p = torch.nn.functional.pad(w, (0, _blocks(cols) * _B - cols, 0, _blocks(rows) * _B - rows))
    p = p.reshape(m, _blocks(rows), _B, _blocks(cols), _B)
    scale = (p.abs().amax((2, 4)) / 448).clamp(min=2.0 ** -126)
    codes = _codes(p, scale[:, :, None, :, None]).reshape(m, _blocks(rows) * _B, -1)[:, :rows, :cols]
    return codes.contiguous(), scale


def _row_parts(rows, n):
    """The e4m3 values and the scales that FP8B rows hold, as views."""
    return [rows[:, :n].view(torch.float8_e4m3fn), rows[:, n:n + 4 * _blocks(n)].view(torch.float32)]


def _row_values(rows, n):
    """FP8B rows [..., row bytes] as 32-bit values [..., n]."""
    scale = rows[..., n:n + 4 * _blocks(n)].contiguous().view(torch.float32)
    return rows[..., :n].view(torch.float8_e4m3fn).float().mul_(scale.repeat_interleave(_B, dim=-1)[..., :n])


def _weight_values(codes, scale):
    """Codes [matrices, rows, cols] and their blocks' scales as 32-bit values."""
    v = codes.float()
    for i in range(scale.shape[1]):
        v[:, i * _B:(i + 1) * _B] *= scale[:, i, None].repeat_interleave(_B, dim=-1)[..., :v.shape[2]]
    return v


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _counts(c, g):
    """Rows of each (expert, source rank): distinct top-k choices of every token, some masked."""
    R, E, K, tokens = c["R"], c["E"], c["K"], c["tokens"]
    p = (torch.arange(E, device="cuda") + 1.0) ** -c["zipf"]
    # Gumbel keys: the K largest are K draws without replacement from p
    key = p.log() - torch.empty(R * tokens, E, device="cuda").exponential_(generator=g).log()
    idx = key.topk(K, dim=1).indices
    kept = torch.rand(R * tokens, K, generator=g, device="cuda") >= c["mask"]
    src = torch.arange(R, device="cuda").repeat_interleave(tokens)[:, None]
    return torch.bincount((idx * R + src)[kept], minlength=E * R).reshape(E, R)


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    s = {"case": c}
    if c["op"] == "router":
        rows, E, K = c["rows"], c["experts"], c["topk"]
        s["logits"] = _normal(g, rows, E).to(_T[c["dtype"]])
        s["bias"] = 0.1 * _normal(g, E) if c["bias"] else None
        s["active"] = (torch.rand(rows, generator=g, device="cuda") >= c["idle"]).to(torch.uint8) if c["idle"] else None
        s["idx"] = torch.empty(rows, K, dtype=torch.int64, device="cuda")
        s["w"] = torch.empty(rows, K, device="cuda")
    elif c["op"] == "rows":
        t, n = _T[c["dtype"]], c["hidden"]
        s["x"] = _normal(g, c["rows"], n).to(t)
        s["residual"] = (4 * _normal(g, c["rows"], n)).to(t) if c["residual"] else None
        s["weight"] = (1 + 0.1 * _normal(g, n)).to(t) if c["norm"] else None
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["out"] = torch.zeros(c["rows"], _row_bytes(n, "fp8b"), dtype=torch.uint8, device="cuda")
        s["views"] = _row_parts(s["out"], n)
    elif c["op"] == "pack":
        m, rows, cols = c["matrices"], c["rows"], c["cols"]
        s["w"] = _normal(g, m, rows, cols, dtype=_T[c["dtype"]]).mul_(cols ** -0.5)
        s["codes"] = torch.zeros(m, rows, cols, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.zeros(m, _blocks(rows), _blocks(cols), device="cuda")
        s["views"] = [s["codes"].view(torch.float8_e4m3fn), s["scale"]]
    else:
        rows, n, parts = c["E"] * c["R"] * c["T"], c["in"], 2 if c["swiglu"] else 1
        s["counts"] = _counts(c, g)
        s["most"] = max(1, int(s["counts"].sum(1).max()))
        s["x"] = torch.empty(rows, _row_bytes(n, "fp8b"), dtype=torch.uint8, device="cuda")
        for a in range(0, rows, 65536):
            b = min(65536, rows - a)
            # a token's values have a size of their own
            s["x"][a:a + b] = _pack_rows(_normal(g, b, n) * (0.5 * _normal(g, b, 1)).exp())
        # gate and up are two matrices, each with its own blocks
        s["w"] = torch.empty(c["E"], parts * c["out"], n, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty(c["E"], parts, _blocks(c["out"]), _blocks(n), device="cuda")
        for e in range(c["E"]):
            codes, s["scale"][e] = _pack_weights(_normal(g, parts, c["out"], n) * n ** -0.5)
            s["w"][e] = codes.view(torch.uint8).reshape(-1, n)
        if c["out_type"] == "fp8b":
            s["y"] = torch.zeros(rows, _row_bytes(c["out"], "fp8b"), dtype=torch.uint8, device="cuda")
            s["views"] = _row_parts(s["y"], c["out"])
        else:
            s["y"] = torch.zeros(rows, c["out"], dtype=_T[c["out_type"]], device="cuda")
            s["views"] = [s["y"]]
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _router(c, s):
    l = s["logits"].float()
    if c["scoring"] == "sigmoid":
        score = 1 / (1 + (-l).exp())
        key = score
    else:
        e = (l - l.amax(-1, keepdim=True)).exp()
        score = e / e.sum(-1, keepdim=True)
        key = l
    if c["bias"]:
        key = key + s["bias"]
    grouped = key.reshape(len(key), c["groups"], -1)
    if c["top2"]:
        best = grouped.sort(dim=-1, descending=True).values
        of_group = best[..., 0] + best[..., 1]
    else:
        of_group = grouped.amax(-1)
    kept = of_group.sort(dim=-1, descending=True, stable=True).indices[:, :c["kept"]]
    on = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, kept, True)
    key = torch.where(on[..., None], grouped, -torch.inf).reshape(key.shape)
    idx = key.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk"]]
    w = score.gather(1, idx)
    w = w * (2.5 / w.sum(-1, keepdim=True)) if c["renorm"] else w * 2.5
    if s["active"] is not None:
        on = s["active"][:, None] != 0
        idx, w = torch.where(on, idx, -1), torch.where(on, w, 0.0)
    s["idx"].copy_(idx)
    s["w"].copy_(w)
    return [s["idx"], s["w"]]


def _rows(c, s):
    v = s["x"].float()
    if c["residual"]:
        s["sum"].copy_(v + s["residual"].float())
        v = s["sum"].float()
    if c["norm"]:
        v = v * (1 / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt()) * s["weight"].float()
    s["out"].copy_(_pack_rows(v))
    return s["views"] + ([s["sum"]] if c["residual"] else [])


def _pack(c, s):
    codes, scale = _pack_weights(s["w"].float())
    s["codes"].copy_(codes.view(torch.uint8))
    s["scale"].copy_(scale)
    return s["views"]


def _table(c, counts, most):
    """Row of x of each expert's j-th received row [E, most], and which of them exist."""
    E, R, T = c["E"], c["R"], c["T"]
    slot = torch.arange(T, device="cuda")
    before = counts.cumsum(1) - counts
    place = torch.where(slot < counts[..., None], before[..., None] + slot, most).reshape(E, R * T)
    rows = torch.arange(E * R * T, device="cuda").reshape(E, R * T)
    table = torch.zeros(E, most + 1, dtype=torch.int64, device="cuda").scatter_(1, place, rows)[:, :most]
    return table, torch.arange(most, device="cuda") < counts.sum(1, keepdim=True)


def _product(c, s):
    table, there = _table(c, s["counts"], s["most"])
    x = _row_values(s["x"][table], c["in"])
    codes, scale = s["w"].view(torch.float8_e4m3fn), s["scale"]
    if c["swiglu"]:
        gate, up = (torch.bmm(x, _weight_values(p, q).transpose(1, 2))
                    for p, q in zip(codes.chunk(2, dim=1), scale.unbind(1)))
        r = gate / (1 + (-gate).exp()) * up
    else:
        r = torch.bmm(x, _weight_values(codes, scale[:, 0]).transpose(1, 2))
    r = r[there]
    s["y"][table[there]] = _pack_rows(r) if c["out_type"] == "fp8b" else r.to(s["y"].dtype)
    return s["views"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"router": _router, "rows": _rows, "pack": _pack, "product": _product}[c["op"]](c, s)
    from combine_routing_count_prefix_gb300 import llmoe
    code = llmoe.ROW_DTYPE_CODES
    if c["op"] == "router":
        flags = (llmoe.LLMOE_ROUTER_RENORM if c["renorm"] else 0) | (llmoe.LLMOE_ROUTER_GROUP_TOP2 if c["top2"] else 0)
        scoring = llmoe.LLMOE_SCORE_SIGMOID if c["scoring"] == "sigmoid" else llmoe.LLMOE_SCORE_SOFTMAX
        llmoe.llmoe_group_router(s["logits"], s["bias"], s["active"], s["idx"], s["w"], c["rows"], c["experts"],
                                 c["topk"], c["groups"], c["kept"], code[c["dtype"]], scoring, flags, 2.5)
        return [s["idx"], s["w"]]
    if c["op"] == "rows":
        if c["norm"]:
            llmoe.llmoe_add_rmsnorm(s["x"], s["residual"], s["weight"], 1e-6, s["sum"], s["out"], c["rows"],
                                    c["hidden"], code[c["dtype"]], code["fp8b"])
        else:
            llmoe.llmoe_pack_fp8b(s["x"], s["out"], c["rows"], c["hidden"], code[c["dtype"]])
        return s["views"] + ([s["sum"]] if c["residual"] else [])
    if c["op"] == "pack":
        llmoe.llmoe_pack_fp8b_weights(s["w"], s["codes"], s["scale"], c["matrices"], c["rows"], c["cols"],
                                      code[c["dtype"]])
        return s["views"]
    bs = llmoe.geometry(num_max_tokens=c["T"], num_ranks=c["R"], num_experts=c["E"])
    llmoe.llmoe_expert_product_fp8b(s["x"], s["w"], s["scale"], s["y"], s["counts"], c["in"], c["out"],
                                    code[c["out_type"]], llmoe.LLMOE_PRODUCT_SWIGLU if c["swiglu"] else 0, bs)
    return s["views"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "router":
        return {"bytes": c["rows"] * (c["experts"] * _BYTES[c["dtype"]] + 12 * c["topk"]) + 4 * c["experts"],
                "flops": 8 * c["rows"] * c["experts"]}
    if c["op"] == "rows":
        row = _row_bytes(c["hidden"], c["dtype"])
        return {"bytes": c["rows"] * (row * (3 if c["residual"] else 1) + _row_bytes(c["hidden"], "fp8b")) + row,
                "flops": 6 * c["rows"] * c["hidden"]}
    if c["op"] == "pack":
        n = c["matrices"] * c["rows"] * c["cols"]
        return {"bytes": n * (_BYTES[c["dtype"]] + 1) + 4 * c["matrices"] * _blocks(c["rows"]) * _blocks(c["cols"]),
                "flops": 2 * n}
    E, K, tokens = c["E"], c["K"], c["R"] * c["tokens"]
    rows = tokens * K * (1 - c["mask"])
    p = [(e + 1) ** -c["zipf"] for e in range(E)]
    # experts that some token chooses, about: a token's K choices hit an expert of share p K times as often as one
    hit = sum(1 - (1 - min(1.0, K * q / sum(p))) ** (tokens * (1 - c["mask"])) for q in p)
    parts = 2 if c["swiglu"] else 1
    weights = parts * (c["out"] * c["in"] + 4 * _blocks(c["out"]) * _blocks(c["in"]))
    return {"bytes": rows * (_row_bytes(c["in"], "fp8b") + _row_bytes(c["out"], c["out_type"])) + hit * weights
            + 8 * E * c["R"],
            "flops": 2 * rows * c["in"] * parts * c["out"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_blocks(v):
    """64-bit values [rows, n] as what their FP8B rows would hold without rounding: value / scale, and the scales."""
    parts = v.split(_B, dim=1)
    scale = torch.stack([p.abs().amax(1) / 448 for p in parts], 1).clamp(min=2.0 ** -126)
    return [torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1), scale]


def _exact_codes(codes):
    """The 64-bit values of e4m3 codes, from their bits."""
    b = torch.arange(256, device="cuda")
    e, m = b >> 3 & 15, (b & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(b >= 128, -mag, mag)[codes.int()]


def _exact_rows(rows, n):
    scale = rows[:, n:n + 4 * _blocks(n)].contiguous().view(torch.float32).double()
    return _exact_codes(rows[:, :n]) * torch.repeat_interleave(scale, _B, dim=1)[:, :n]


def _exact_weights(codes, scale):
    r, n = codes.shape
    at = torch.arange(r, device="cuda") // _B, torch.arange(n, device="cuda") // _B
    return _exact_codes(codes) * scale.double()[at[0][:, None], at[1][None, :]]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "router":
        l = s["logits"].double()
        if c["scoring"] == "sigmoid":
            score = torch.sigmoid(l)
            key = score.float()
        else:
            score = torch.softmax(l, -1)
            key = s["logits"].float()
        if c["bias"]:
            key = key + s["bias"]
        of = torch.topk(key.unflatten(1, (c["groups"], -1)), 2 if c["top2"] else 1, dim=-1).values.sum(-1)
        left = torch.argsort(of, dim=-1, descending=True, stable=True)[:, c["kept"]:]
        size = c["experts"] // c["groups"]
        out = (left[:, :, None] * size + torch.arange(size, device="cuda")).flatten(1)
        key = key.scatter(1, out, -torch.inf)
        idx = torch.argsort(key, dim=-1, descending=True, stable=True)[:, :c["topk"]]
        w = torch.take_along_dim(score, idx, 1) * 2.5
        if c["renorm"]:
            w = 2.5 * w / w.sum(-1, keepdim=True)
        if s["active"] is not None:
            w[s["active"] == 0] = 0.0
        return [None, w]
    if c["op"] == "rows":
        v, first = s["x"].double(), []
        if c["residual"]:
            total = v + s["residual"].double()
            first = [total]
            v = total.to(_T[c["dtype"]]).double()  # the definition norms the stored sum
        if c["norm"]:
            v = v * torch.rsqrt((v * v).sum(-1, keepdim=True) / c["hidden"] + 1e-6) * s["weight"].double()
        return _exact_blocks(v) + first
    if c["op"] == "pack":
        codes = torch.empty(s["w"].shape, dtype=torch.float32, device="cuda")
        scale = torch.empty(s["scale"].shape, dtype=torch.float64, device="cuda")
        for i in range(scale.shape[1]):
            for j in range(scale.shape[2]):
                at = (slice(None), slice(i * _B, (i + 1) * _B), slice(j * _B, (j + 1) * _B))
                v = s["w"][at].double()
                scale[:, i, j] = (v.abs().amax((1, 2)) / 448).clamp(min=2.0 ** -126)
                codes[at] = (v / scale[:, i, j, None, None]).float()
        return [codes, scale]
    E, R, T, out = c["E"], c["R"], c["T"], c["out"]
    counts = s["counts"].tolist()
    if E * R * T * out > 1 << 31:
        return None
    parts = [torch.zeros(E * R * T, out, dtype=torch.float64, device="cuda")]
    if c["out_type"] == "fp8b":
        parts.append(torch.zeros(E * R * T, _blocks(out), dtype=torch.float64, device="cuda"))
    for e in range(E):
        at = [torch.arange(n, device="cuda") + (e * R + src) * T for src, n in enumerate(counts[e]) if n]
        if not at:
            continue
        at = torch.cat(at)
        x = _exact_rows(s["x"][at], c["in"])
        r = [x @ _exact_weights(s["w"][e, i * out:(i + 1) * out], s["scale"][e, i]).T for i in range(s["scale"].shape[1])]
        r = r[0] * torch.sigmoid(r[0]) * r[1] if c["swiglu"] else r[0]
        for p, v in zip(parts, _exact_blocks(r) if c["out_type"] == "fp8b" else [r]):
            p[at] = v
    return parts
