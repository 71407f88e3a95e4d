/*
 * llmoe_block.h -- C ABI of the operators around the dispatch and combine of
 * one MoE block (libllmoe.so, GB300 / sm_103a): the norm that makes the rows
 * to dispatch, the router that makes topk_idx and topk_w, and the experts'
 * matrix products over the received rows.
 *
 * The conventions are llmoe.h's: device pointers into the caller's memory, no
 * allocation and no synchronisation, work enqueued on `stream`, argument
 * checks on the host before any launch, llmoe_status_t results.  No call
 * needs a workspace.
 *
 * One block, with 8-bit rows on the way to the experts:
 *   llmoe_add_rmsnorm(x, residual, w, eps, residual, rows, ..., LLMOE_DTYPE_MX8)
 *   llmoe_topk_router(logits, ..., topk_idx, topk_w, ...)
 *   llmoe_dispatch_unpack(rows, topk_idx, recv_x, recv_src, &bs)
 *   llmoe_expert_product(recv_x, w_gate_up, h, NULL, ..., LLMOE_PRODUCT_SWIGLU, &bs)
 *   llmoe_expert_product(h, w_down, y, NULL, ..., 0, &bs)
 *   llmoe_combine(y, topk_idx, topk_w, out, &bs_out)
 */
#ifndef LLMOE_BLOCK_H_
#define LLMOE_BLOCK_H_

#include "llmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The row type MX8: 8-bit values with a scale for each 32 of them.  A row of n
 * values (n a multiple of 32) is n e4m3 codes, then n / 32 e8m0 scale codes (a
 * code c is the scale 2^(c - 127)), then zeros up to a multiple of 16 bytes:
 * llmoe_row_bytes(n, LLMOE_DTYPE_MX8) bytes.  A value is its code times its
 * group's scale.  The library writes the smallest power-of-two scale at which
 * no value of the group exceeds 448, e4m3's largest (at least 2^-126), and
 * rounds each quotient to nearest even; a group that holds an infinity or a
 * NaN gets the NaN scale 255.
 * MX8 rows travel through the dispatch unchanged, as the rows of a bf16
 * buffer set of hidden = llmoe_row_bytes(n, LLMOE_DTYPE_MX8) / 2.  The calls
 * of llmoe.h do not take MX8 as a payload type. */
#define LLMOE_DTYPE_MX8 3

/* Largest `hidden` of llmoe_add_rmsnorm and llmoe_pack_mx8. */
#define LLMOE_MAX_ROW_VALUES 32768

/* Bytes of one row of `n` values of type `dtype` (LLMOE_DTYPE_*, MX8 among
 * them): 0 when n < 1, when the type is unknown, when n is not a multiple of
 * 32 for MX8, or when a row of another type is not a multiple of 16 bytes. */
LLMOE_API size_t llmoe_row_bytes(int n, int dtype);

/* Rows of BF16, FP16 or FP32 values as MX8 rows (a model's weights, once, or
 * activations that no norm precedes).
 *   x    device T [rows][hidden], 16-byte aligned; T per dtype.
 *   out  device MX8 rows [rows], 16-byte aligned, must not overlap x.
 * hidden: a multiple of 32, at most LLMOE_MAX_ROW_VALUES. */
LLMOE_API int llmoe_pack_mx8(const void* x, void* out, int64_t rows, int hidden, int dtype, llmoe_stream_t stream);

/* Residual addition and root-mean-square norm:
 *   h = T(x + residual)                       (residual NULL: h = x)
 *   residual_out = h                          (residual_out NULL: not written)
 *   v = h * (1 / sqrt(mean(h^2) + eps)) * weight   in fp32
 *   out = T(v), or v as MX8 rows.
 * The norm is that of the rounded sum, the value the next block reads back.
 *   x, residual, residual_out  device T [rows][hidden]; T per dtype.
 *   weight     device T [hidden].
 *   out        device rows [rows] of out_dtype: dtype or LLMOE_DTYPE_MX8.
 * All pointers 16-byte aligned.  residual_out may be x or residual, and out
 * may be x (out_dtype == dtype); no other overlap.  hidden: a row of T is a
 * multiple of 16 bytes (and hidden of 32 for MX8), at most
 * LLMOE_MAX_ROW_VALUES.  eps >= 0.  rows may be 0. */
LLMOE_API int llmoe_add_rmsnorm(const void* x, const void* residual, const void* weight, float eps,
                                void* residual_out, void* out, int64_t rows, int hidden, int dtype, int out_dtype,
                                llmoe_stream_t stream);

/* llmoe_topk_router scoring */
#define LLMOE_SCORE_SIGMOID 0 /* score = 1 / (1 + exp(-l)), key = score + bias */
#define LLMOE_SCORE_SOFTMAX 1 /* score = softmax(l) over the row's experts that can be chosen, key = l + bias */
/* llmoe_topk_router flags */
#define LLMOE_ROUTER_RENORM 1u /* divide the chosen scores by their sum */

/* Router: each row's num_topk experts of largest key, in descending order of
 * key, equal keys by ascending expert; their weights are scale * score (with
 * LLMOE_ROUTER_RENORM, scale * (score / the sum of the row's chosen scores); 0
 * where that sum is 0).  Scores, keys and sums are fp32: a sigmoid below 2^-128
 * is 0.  A renormalised softmax is taken over the chosen alone, which is the
 * same, so that an unchosen expert far above them does not make their scores 0.
 *   logits    device T [rows][num_experts]; T per dtype (BF16, FP16, FP32).
 *   bias      device fp32 [num_experts], or NULL.
 *   active    device uint8 [rows], or NULL: rows with 0 choose nothing.
 *   topk_idx  device int64 [rows][num_topk] out, as llmoe_dispatch takes it.
 *   topk_w    device fp32 [rows][num_topk] out, as llmoe_combine takes it.
 * An expert whose logit or key is NaN or -infinity cannot be chosen and has
 * score 0; where fewer than num_topk can, the remaining entries are -1 with
 * weight 0.  Softmax: such experts are not in its sum; logits of +infinity share
 * the whole weight.
 * LLMOE_FLAG_INPUTS_READY on the dispatch or combine that takes them needs
 * another call of this header between the router and that call (the experts'
 * products, for a combine): what starts behind such a call finds all before
 * it complete, where the calls of llmoe.h may start while it is at work.
 * topk_idx and topk_w must overlap neither each other nor an input.
 * 1 <= num_topk <= min(num_experts, LLMOE_MAX_TOPK), num_experts <=
 * LLMOE_MAX_EXPERTS.  rows may be 0. */
LLMOE_API int llmoe_topk_router(const void* logits, const float* bias, const uint8_t* active, int64_t* topk_idx,
                                float* topk_w, int64_t rows, int num_experts, int num_topk, int dtype, int scoring,
                                uint32_t flags, float scale, llmoe_stream_t stream);

/* llmoe_expert_product flags */
#define LLMOE_PRODUCT_SWIGLU 1u /* w holds gate and up; y = silu(x gate^T) * (x up^T) */

/* Matrix products grouped by expert over the received rows: for every expert
 * e, source rank src and slot < counts[e][src], with r = (e * R + src) * T +
 * slot (the row order of llmoe_unpack's recv_x and llmoe_combine's y; T =
 * bs->num_max_tokens),
 *   y[r][:] = x[r][:] w[e]^T       summed in fp32, rounded once to out_dtype;
 * with LLMOE_PRODUCT_SWIGLU w[e] is [gate; up], 2 * out_features rows, and
 *   y[r][:] = silu(x[r] gate^T) * (x[r] up^T),  silu(a) = a / (1 + exp(-a)), in fp32.
 * (Where y is of 16 or 8 bits, exp and the quotient are the hardware's: within
 * 4 + |a| / 2 units of the last fp32 place, which y's rounding covers.)
 * Other rows of y are not written.  Unreceived rows of x, whatever they hold,
 * do not touch the result.
 *   x       device rows of dtype [E * R * T], in_features values each.
 *   w       device rows of dtype [E][out_features, or 2 * out_features with
 *           LLMOE_PRODUCT_SWIGLU], in_features values each.
 *   y       device rows of out_dtype [E * R * T], out_features values each;
 *           must not overlap x or w.
 *   counts  device int64 [E][R], llmoe_route's counts; or NULL: the recv-count
 *           words of buffer set bs->set, as a dispatch leaves them.  Counts
 *           are taken as clamped to [0, T]; outside it validate mode reports
 *           LLMOE_DEV_SLOT_RANGE.
 *   dtype   LLMOE_DTYPE_BF16, _FP16 or _MX8 (there is no fp32 product: the
 *           tensor cores have no fp32 operands).
 *   out_dtype  dtype, or LLMOE_DTYPE_FP32; for MX8 operands BF16, FP16 or
 *           FP32, and MX8 with LLMOE_PRODUCT_SWIGLU.
 *   bs      geometry: num_max_tokens, num_ranks, num_experts, and err; with
 *           counts NULL also base, rank_stride, hidden, dtype and set.
 * Every wait inside the kernel is bounded (about a second); one that expires
 * leaves its rows unwritten and validate mode reports LLMOE_DEV_TIMEOUT.
 * x, w, y 16-byte aligned; llmoe_row_bytes(in_features, dtype) and
 * llmoe_row_bytes(out_features, out_dtype) not 0; out_features a multiple of
 * 8 with LLMOE_PRODUCT_SWIGLU; E * R * T < 2^31. */
LLMOE_API int llmoe_expert_product(const void* x, const void* w, void* y, const int64_t* counts, int in_features,
                                   int out_features, int dtype, int out_dtype, uint32_t flags,
                                   const llmoe_buf_set_t* bs, llmoe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LLMOE_BLOCK_H_ */
