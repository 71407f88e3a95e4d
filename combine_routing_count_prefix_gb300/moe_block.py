"""One MoE block over the library's calls: norm, router, dispatch, expert
products, combine.

``MoEBlock`` holds what a serving program keeps for one block (rank buffers,
weights laid out once, activations) and runs a micro-batch of tokens through
it:

    residual += x; rows = norm(residual)            llmoe_add_rmsnorm
    logits = rows @ router_weight.T                 llmoe_expert_product (one "expert" holding every token)
    topk_idx, topk_w = route(logits)                llmoe_topk_router or llmoe_group_router
    recv_x, counts = dispatch(rows, topk_idx)       llmoe_dispatch_unpack
    h = swiglu(recv_x @ gate_up.T)                  llmoe_expert_product
    y = h @ down.T                                  llmoe_expert_product
    out = combine(y, topk_idx, topk_w)              llmoe_combine

With ``rows="mx8"`` the dispatched rows, the expert weights and h are 8-bit
rows with a scale for each 32 values: half the bytes of a decode step.  With
``rows="fp8b"`` rows have a fp32 scale for each 128 values and weights one for
each 128 x 128 block, as checkpoints hold them (llmoe_expert_product_fp8b).  The
router then still reads rows of the block's own type.  Where its experts come in
groups, llmoe_group_router routes.

This module only orders calls; every step runs in the library's kernels, on
the current stream, and one call of ``forward`` can be captured in a CUDA
graph.
"""
from __future__ import annotations

import torch

from . import llmoe

_TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}


def pack_mx8(w: torch.Tensor) -> torch.Tensor:
    """Values [..., n] as MX8 rows [..., row bytes] (uint8)."""
    n = w.shape[-1]
    code = {torch.bfloat16: llmoe.LLMOE_DTYPE_BF16, torch.float16: llmoe.LLMOE_DTYPE_FP16,
            torch.float32: llmoe.LLMOE_DTYPE_FP32}[w.dtype]
    nbytes = llmoe.llmoe_row_bytes(n, llmoe.LLMOE_DTYPE_MX8)
    if nbytes == 0:
        raise ValueError(f"MX8 rows hold multiples of 32 values, not {n}")
    out = torch.empty(*w.shape[:-1], nbytes, dtype=torch.uint8, device=w.device)
    llmoe.llmoe_pack_mx8(w.contiguous(), out, w.numel() // n, n, code)
    return out


def pack_fp8b_weights(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Matrices [..., rows, cols] as e4m3 codes (uint8, the same shape) and the fp32
    scales [..., ceil(rows / 128), ceil(cols / 128)] of their 128 x 128 blocks."""
    code = {torch.bfloat16: llmoe.LLMOE_DTYPE_BF16, torch.float16: llmoe.LLMOE_DTYPE_FP16,
            torch.float32: llmoe.LLMOE_DTYPE_FP32}.get(w.dtype)
    if code is None:
        raise ValueError(f"weights are bf16, fp16 or fp32, not {w.dtype}")
    if w.dim() < 2 or 0 in w.shape[-2:]:
        raise ValueError(f"no matrices: {tuple(w.shape)}")
    rows, cols = w.shape[-2:]
    if cols % 16:
        raise ValueError(f"rows of {cols} codes are not whole 16 bytes")
    codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    scales = torch.empty(*w.shape[:-2], _blocks(rows), _blocks(cols), dtype=torch.float32, device=w.device)
    llmoe.llmoe_pack_fp8b_weights(w.contiguous(), codes, scales, w.numel() // (rows * cols), rows, cols, code)
    return codes, scales


def _blocks(n: int) -> int:
    return -(-n // llmoe.LLMOE_FP8B_BLOCK)


def _tensor(name: str, t: torch.Tensor, shape: tuple, dtypes: tuple, device: torch.device, laid_out: bool = True) -> None:
    """The calls take addresses: what lies behind one is checked here."""
    if t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype} {list(t.shape)}, not {dtypes[0]} {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on device {t.device}, the block on {device}")
    if laid_out and not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")


def _weight(name: str, t: torch.Tensor, shape: tuple, dtypes: tuple, device: torch.device, laid_out: bool = True) -> None:
    """A weight, which a call behind others must not refuse.  What is not laid out is
    packed, from a copy where it is not contiguous."""
    _tensor(name, t, shape, dtypes, device, laid_out)
    if t.is_contiguous() and t.data_ptr() % 16:
        raise ValueError(f"{name} is not 16-byte aligned")


class MoEBlock:
    """
    num_max_tokens  T: tokens per rank a call may have
    norm_weight     [H]
    router_weight   [E, H], E a multiple of 4 (fp32 logits rows of whole 16 bytes);
                    router_bias [E] fp32 or None (added to what is chosen by, the sigmoids or,
                    with softmax, the logits; not to the weights)
    gate_up         [E, 2 I, H], gate rows first; down [E, H, I].  These four start at 16-byte
                    boundaries; gate_up and down that are packed may be of any layout
    dtype           "bf16" or "fp16": x, weights and output (with rows="mx8"
                    gate_up and down, which are packed, may be bf16, fp16 or fp32;
                    with rows="fp8b" the same, or e4m3 codes with gate_up_scale and
                    down_scale)
    rows            "same": rows and experts in dtype; "mx8": 8-bit rows and expert weights;
                    "fp8b": the same with scales by blocks of 128
    num_groups      groups of experts, of which a token chooses from kept_groups (all of
                    them, unless given); group_top2: a group's score is the sum of its two
                    largest keys, else its largest
    renorm          a token's weights are scale * score / (the sum of its chosen scores), else
                    scale * score: what a softmax over all experts leaves to the chosen
    gate_up_scale   [E, 2, ceil(I / 128), ceil(H / 128)] fp32, with gate_up as codes (uint8 or
                    float8_e4m3fn); down_scale [E, ceil(H / 128), ceil(I / 128)]
    """

    def __init__(self, num_max_tokens: int, num_ranks: int, num_topk: int, norm_weight: torch.Tensor,
                 router_weight: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor,
                 router_bias: torch.Tensor | None = None, dtype: str = "bf16", rows: str = "same",
                 eps: float = 1e-6, scale: float = 1.0, scoring: int = llmoe.LLMOE_SCORE_SIGMOID, err=None,
                 num_groups: int = 1, kept_groups: int | None = None, group_top2: bool = False,
                 gate_up_scale: torch.Tensor | None = None, down_scale: torch.Tensor | None = None,
                 renorm: bool = True):
        if rows not in ("same", "mx8", "fp8b"):
            raise ValueError(f'rows is "same", "mx8" or "fp8b", not {rows!r}')
        if dtype not in _TORCH:
            raise ValueError(f'dtype is "bf16" or "fp16", not {dtype!r}')
        for name, w, dims in (("router_weight", router_weight, 2), ("down", down, 3)):
            if w.dim() != dims:
                raise ValueError(f"{name} has {w.dim()} dimensions, not {dims}")
        self.E, self.H = router_weight.shape
        self.I = down.shape[2]
        self.T, self.R, self.K = num_max_tokens, num_ranks, num_topk
        E, H, I = self.E, self.H, self.I
        self.own, self.device = own, dev = (_TORCH[dtype],), norm_weight.device
        packed = (*own, torch.bfloat16, torch.float16, torch.float32) if rows != "same" else own
        coded = gate_up_scale is not None or down_scale is not None
        if coded:
            if rows != "fp8b" or gate_up_scale is None or down_scale is None:
                raise ValueError('gate_up_scale and down_scale are given together, with rows="fp8b"')
            _tensor("gate_up_scale", gate_up_scale, (E, 2, _blocks(I), _blocks(H)), (torch.float32,), dev)
            _tensor("down_scale", down_scale, (E, _blocks(H), _blocks(I)), (torch.float32,), dev)
            packed = (torch.uint8, torch.float8_e4m3fn)
        _weight("norm_weight", norm_weight, (H,), own, dev)
        _weight("router_weight", router_weight, (E, H), own, dev)
        _weight("gate_up", gate_up, (E, 2 * I, H), packed, dev, rows == "same" or coded)
        _weight("down", down, (E, H, I), packed, dev, rows == "same" or coded)
        if router_bias is not None:
            _tensor("router_bias", router_bias, (E,), (torch.float32,), dev)
        if self.T < 1:
            raise ValueError(f"num_max_tokens is {self.T}")
        if self.R < 1 or E % self.R:
            raise ValueError(f"num_ranks is {self.R}: {E} experts do not divide over them")
        if not 1 <= self.K <= min(E, llmoe.LLMOE_MAX_TOPK):
            raise ValueError(f"num_topk is {self.K} of {E} experts, at most {llmoe.LLMOE_MAX_TOPK}")
        self.G, self.kept = num_groups, num_groups if kept_groups is None else kept_groups
        if not 1 <= self.G <= llmoe.LLMOE_MAX_GROUPS or E % self.G:
            raise ValueError(f"num_groups is {self.G} of {E} experts, at most {llmoe.LLMOE_MAX_GROUPS}")
        if not 1 <= self.kept <= self.G or self.K > E // self.G * self.kept:
            raise ValueError(f"kept_groups is {self.kept} of {self.G}, num_topk {self.K}")
        if scoring not in (llmoe.LLMOE_SCORE_SIGMOID, llmoe.LLMOE_SCORE_SOFTMAX):
            raise ValueError(f"scoring is {scoring!r}")
        if group_top2 and scoring != llmoe.LLMOE_SCORE_SIGMOID:
            raise ValueError("group_top2 goes with sigmoid scores")
        self.renorm_flag = llmoe.LLMOE_ROUTER_RENORM if renorm else 0
        self.group_flag = llmoe.LLMOE_ROUTER_GROUP_TOP2 if group_top2 else 0
        for width in (H, I):
            if llmoe.llmoe_row_bytes(width, llmoe.ROW_DTYPE_CODES[dtype if rows == "same" else rows]) == 0:
                raise ValueError(f"a hidden size of {width}: a row is whole 16 bytes, MX8 rows multiples of 32 values, "
                                 "FP8B rows of 16")
        self.eps, self.scale, self.scoring = eps, scale, scoring
        self.code = llmoe.DTYPE_CODES[dtype]
        self.row_code = self.code if rows == "same" else llmoe.ROW_DTYPE_CODES[rows]
        self.norm_weight, self.router_weight, self.router_bias = norm_weight, router_weight, router_bias
        self.gate_up = pack_mx8(gate_up) if rows == "mx8" else gate_up
        self.down = pack_mx8(down) if rows == "mx8" else down
        self.gate_up_scale, self.down_scale = gate_up_scale, down_scale
        if rows == "fp8b" and not coded:
            self.gate_up, self.gate_up_scale = pack_fp8b_weights(gate_up.reshape(E, 2, I, H))
            self.down, self.down_scale = pack_fp8b_weights(down)
        t = _TORCH[dtype]
        tokens, received = self.R * self.T, self.E * self.R * self.T
        row = llmoe.llmoe_row_bytes(self.H, self.row_code)
        # what is dispatched: rows of dtype, or 8-bit rows as a 16-bit payload of their bytes
        self.rb_dispatch = llmoe.RankBuffers(self.T, row // 2, self.R, self.E, device=dev, dtype=dtype)
        self.rb_combine = llmoe.RankBuffers(self.T, self.H, self.R, self.E, device=dev, dtype=dtype)
        self.err = err
        self.xn = torch.empty(tokens, self.H, dtype=t, device=dev)
        self.rows = self.xn if rows == "same" else torch.empty(tokens, row, dtype=torch.uint8, device=dev)
        self.logits = torch.empty(tokens, self.E, dtype=torch.float32, device=dev)
        self.topk_idx = torch.empty(tokens, self.K, dtype=torch.int64, device=dev)
        self.topk_w = torch.empty(tokens, self.K, dtype=torch.float32, device=dev)
        self.recv_x = torch.empty(received, row // 2, dtype=t, device=dev)
        self.recv_src = torch.empty(received, dtype=torch.int32, device=dev)
        self.h = torch.empty(received, llmoe.llmoe_row_bytes(self.I, self.row_code), dtype=torch.uint8, device=dev)
        self.y = torch.empty(received, self.H, dtype=t, device=dev)
        # the router product's one count, for every number of tokens a call may have
        self.token_counts = torch.arange(self.T + 1, dtype=torch.int64, device=dev) * self.R

    def forward(self, x: torch.Tensor, residual: torch.Tensor, out: torch.Tensor,
                active: torch.Tensor | None = None) -> torch.Tensor:
        """x, residual, out [R, tokens, H]: residual becomes residual + x, out
        the block's output (to be added to the residual by the next block).
        active [R, tokens] uint8 or bool: tokens with 0 are routed nowhere and give 0."""
        if x.dim() != 3:
            raise ValueError(f"x has {x.dim()} dimensions, not 3")
        R, n, H, E = x.shape[0], x.shape[1], self.H, self.E
        if R != self.R or n > self.T:
            raise ValueError(f"x holds {R} ranks of {n} tokens, the block {self.R} of at most {self.T}")
        if E % 4:
            raise ValueError(f"{E} experts are not a multiple of 4")
        shape, own, dev = (R, n, H), self.own, self.device
        _tensor("x", x, shape, own, dev)
        _tensor("residual", residual, shape, own, dev)
        _tensor("out", out, shape, own, dev)
        if active is not None:
            _tensor("active", active, (R, n), (torch.uint8, torch.bool), dev)
        if (x.data_ptr() | residual.data_ptr() | out.data_ptr()) % 16:
            raise ValueError("x, residual and out are 16-byte aligned")
        if abs(out.data_ptr() - residual.data_ptr()) < 2 * R * n * H:
            raise ValueError("out and residual overlap")
        tokens = R * n
        L, code, row_code = llmoe, self.code, self.row_code
        if row_code == code:
            L.llmoe_add_rmsnorm(x, residual, self.norm_weight, self.eps, residual, self.xn, tokens, H, code, code)
        else:
            L.llmoe_add_rmsnorm(x, residual, self.norm_weight, self.eps, residual, self.rows, tokens, H, code, row_code)
            L.llmoe_add_rmsnorm(residual, None, self.norm_weight, self.eps, None, self.xn, tokens, H, code, code)
        # a dense product is one expert that every token was sent to
        L.llmoe_expert_product(self.xn, self.router_weight, self.logits, self.token_counts[n:n + 1], H, E, code,
                               L.LLMOE_DTYPE_FP32, 0, L.geometry(max(1, R * self.T), 1, 1, self.err))
        if self.kept < self.G:
            L.llmoe_group_router(self.logits, self.router_bias, active, self.topk_idx, self.topk_w, tokens, E, self.K,
                                 self.G, self.kept, L.LLMOE_DTYPE_FP32, self.scoring,
                                 self.renorm_flag | self.group_flag, self.scale)
        else:
            L.llmoe_topk_router(self.logits, self.router_bias, active, self.topk_idx, self.topk_w, tokens, E, self.K,
                                L.LLMOE_DTYPE_FP32, self.scoring, self.renorm_flag, self.scale)
        d = self.rb_dispatch.buf_set(0, self.K, n, self.err)
        c = self.rb_combine.buf_set(1, self.K, n, self.err)
        L.llmoe_clean(d)
        L.llmoe_dispatch_unpack(self._payload(self.rows), self.topk_idx, self.recv_x, self.recv_src, d)
        if row_code == L.LLMOE_DTYPE_FP8B:
            L.llmoe_expert_product_fp8b(self.recv_x, self.gate_up, self.gate_up_scale, self.h, None, H, self.I, row_code,
                                        L.LLMOE_PRODUCT_SWIGLU, d)
            L.llmoe_expert_product_fp8b(self.h, self.down, self.down_scale, self.y, None, self.I, H, code, 0, d)
        else:
            L.llmoe_expert_product(self.recv_x, self.gate_up, self.h, None, H, self.I, row_code, row_code,
                                   L.LLMOE_PRODUCT_SWIGLU, d)
            L.llmoe_expert_product(self.h, self.down, self.y, None, self.I, H, row_code, code, 0, d)
        L.llmoe_clean(c)
        L.llmoe_combine(self.y, self.topk_idx, self.topk_w, out, c)
        return out

    def _payload(self, rows: torch.Tensor) -> torch.Tensor:
        return rows if rows.dtype != torch.uint8 else rows.view(self.xn.dtype)
