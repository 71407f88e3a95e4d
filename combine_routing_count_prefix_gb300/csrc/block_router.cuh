// block_router.cuh -- what the two routers share: logits, scores, keys and reductions.
#pragma once
#include "block_common.cuh"

namespace {

// A router's arguments: false where they are not valid.
inline bool router_shape(int64_t rows, int num_experts, int num_topk, int dtype, int scoring) {
  return (dtype == LLMOE_DTYPE_BF16 || dtype == LLMOE_DTYPE_FP16 || dtype == LLMOE_DTYPE_FP32) && num_experts >= 1 &&
         num_experts <= LLMOE_MAX_EXPERTS && num_topk >= 1 && num_topk <= LLMOE_MAX_TOPK && num_topk <= num_experts &&
         (scoring == LLMOE_SCORE_SIGMOID || scoring == LLMOE_SCORE_SOFTMAX) && rows >= 0 &&
         rows <= INT64_MAX / 8 / num_experts;
}
inline bool router_memory(const void* logits, const float* bias, const uint8_t* active, int64_t* topk_idx,
                          float* topk_w, int64_t rows, int num_experts, int num_topk, int dtype) {
  const int es = dtype == LLMOE_DTYPE_FP32 ? 4 : 2;
  if (logits == nullptr || topk_idx == nullptr || topk_w == nullptr || !aligned(logits, es) || !aligned(bias, 4) ||
      !aligned(topk_idx, 8) || !aligned(topk_w, 4))
    return false;
  // rows are read and written by many CTAs in no order: no output may be an input
  const uint64_t n = (uint64_t)rows, idx_bytes = n * num_topk * 8, w_bytes = n * num_topk * 4;
  const auto meets = [&](const void* in, uint64_t bytes) {
    return in != nullptr && (overlap(topk_idx, idx_bytes, in, bytes) || overlap(topk_w, w_bytes, in, bytes));
  };
  return !meets(logits, n * num_experts * es) && !meets(bias, (uint64_t)num_experts * 4) && !meets(active, n) &&
         !overlap(topk_idx, idx_bytes, topk_w, w_bytes);
}

__device__ __forceinline__ float load_logit(const void* logits, int dtype, int64_t i) {
  switch (dtype) {
    case LLMOE_DTYPE_BF16: return __bfloat162float(static_cast<const __nv_bfloat16*>(logits)[i]);
    case LLMOE_DTYPE_FP16: return __half2float(static_cast<const __half*>(logits)[i]);
    default: return static_cast<const float*>(logits)[i];
  }
}

__device__ __forceinline__ float sigmoid_score(float l) { return __frcp_rn(1.0f + expf(-l)); }
// 1 / d to the nearest fp32, what __frcp_rn gives, for d from 1 to 2^126 (each of them
// compared by tests/test_gpu_reciprocal.py): the hardware's reciprocal and one step of
// Newton's, whose remainder is exact in a fused multiply-add.  Without the general
// one's other ranges, which a lane's experts would each have in line: one token 2.9 us
// against 3.8, 8192 tokens 9.1 against 9.9.  So 1 / (1 + exp(-v)) for v from -87 on; a
// token with a logit below (-infinity among them) takes the general one.
__device__ __forceinline__ float one_over(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return fmaf(fmaf(-d, r, 1.0f), r, r);
}
// Of a row whose largest logit is top; logits of +infinity are the limit of
// equal large ones.
__device__ __forceinline__ float softmax_score(float l, float top) {
  return top == INFINITY ? (l == INFINITY ? 1.0f : 0.0f) : expf(l - top);
}

// A key as an integer of the same order, 0 where the expert cannot be chosen:
// its logit or key is NaN or -infinity.
__device__ __forceinline__ uint32_t order(float logit, float key) {
  key += 0.0f;  // -0 ranks as +0
  const uint32_t b = __float_as_uint(key);
  return logit > -INFINITY && key > -INFINITY ? ((b & 0x80000000u) ? ~b : (b | 0x80000000u)) : 0u;
}
__device__ __forceinline__ float unorder(uint32_t b) {
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7fffffffu) : ~b);
}

// Reductions over a token's group of W warps; part: W words per use.
template <int W>
struct Group {
  uint32_t* part;
  template <typename T, typename F>
  __device__ __forceinline__ T all(T v, F f) const {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, d));
    if constexpr (W > 1) {
      T* p = reinterpret_cast<T*>(part);
      __syncthreads();
      if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
      __syncthreads();
      v = p[0];
#pragma unroll
      for (int w = 1; w < W; ++w) v = f(v, p[w]);
    }
    return v;
  }
  __device__ __forceinline__ uint32_t max_u32(uint32_t v) const {
    if constexpr (W == 1) return __reduce_max_sync(0xffffffffu, v);
    return all(v, [](uint32_t x, uint32_t y) { return max(x, y); });
  }
  __device__ __forceinline__ uint32_t min_u32(uint32_t v) const {
    if constexpr (W == 1) return __reduce_min_sync(0xffffffffu, v);
    return all(v, [](uint32_t x, uint32_t y) { return min(x, y); });
  }
  __device__ __forceinline__ float max_f(float v) const {
    return all(v, [](float x, float y) { return fmaxf(x, y); });
  }
  __device__ __forceinline__ float sum_f(float v) const {
    return all(v, [](float x, float y) { return x + y; });
  }
};

}  // namespace
