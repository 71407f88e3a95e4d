// block_router.cu -- llmoe_topk_router (include/llmoe_block.h).
//
// A group of one warp (a CTA of eight for more experts than a warp holds in
// registers) owns a token: expert e's key sits in lane e % lanes as a 32-bit
// integer that orders like the float (0: cannot be chosen).  Each of the K
// rounds takes the maximum key and, among its holders, the lowest expert, by
// two warp reductions, so ties go to the lowest index whatever the schedule.
#include "block_common.cuh"

namespace {

struct RouterArgs {
  const void* logits;
  const float* bias;
  const uint8_t* active;
  int64_t* topk_idx;
  float* topk_w;
  int64_t rows;
  int E, K, dtype;
  bool softmax, renorm;
  float scale;
};

__device__ __forceinline__ float load_logit(const RouterArgs& a, int64_t i) {
  switch (a.dtype) {
    case LLMOE_DTYPE_BF16: return __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[i]);
    case LLMOE_DTYPE_FP16: return __half2float(static_cast<const __half*>(a.logits)[i]);
    default: return static_cast<const float*>(a.logits)[i];
  }
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

// W warps per token, V experts per lane.
template <int W, int V>
__global__ void __launch_bounds__(256) router_kernel(RouterArgs a) {
  __shared__ uint32_t part[W];
  release_next_grid();
  wait_prior_grid();
  const Group<W> group{part};
  constexpr int kLanes = 32 * W;
  const int lane = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t first = W == 1 ? ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5 : blockIdx.x;
  const int64_t step = W == 1 ? ((int64_t)gridDim.x * blockDim.x) >> 5 : gridDim.x;
  for (int64_t row = first; row < a.rows; row += step) {
    const bool on = a.active == nullptr || a.active[row] != 0;
    float score[V];
    uint32_t key[V];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + i * kLanes;
      score[i] = on && e < a.E ? load_logit(a, row * a.E + e) : -INFINITY;
      top = fmaxf(top, score[i]);  // a NaN does not count
    }
    if (a.softmax) top = group.max_f(top);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + i * kLanes;
      const float l = score[i];
      const bool can = l > -INFINITY;  // false for a NaN
      float k;
      if (a.softmax) {
        // logits of +infinity are the limit of equal large ones
        score[i] = !can ? 0.0f : top == INFINITY ? (l == INFINITY ? 1.0f : 0.0f) : expf(l - top);
        total += score[i];
        k = l;
      } else {
        score[i] = can ? 1.0f / (1.0f + expf(-l)) : 0.0f;
        k = score[i];
      }
      if (a.bias != nullptr && e < a.E) k += a.bias[e];
      k += 0.0f;  // -0 ranks as +0
      const uint32_t b = __float_as_uint(k);
      key[i] = can && k > -INFINITY ? ((b & 0x80000000u) ? ~b : (b | 0x80000000u)) : 0u;
    }
    if (a.softmax) {
      total = group.sum_f(total);
#pragma unroll
      for (int i = 0; i < V; ++i) score[i] = total > 0.0f ? score[i] / total : 0.0f;
    }
    int my_idx = -1;  // lane k of the first warp keeps the k-th choice
    float my_score = 0.0f, sum = 0.0f;
    for (int k = 0; k < a.K; ++k) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) best = max(best, key[i]);
      best = group.max_u32(best);
      if (best == 0) break;  // nothing left to choose: uniform over the group
      uint32_t at = 0xffffffffu;
      float s = 0.0f;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (key[i] == best) at = lane + i * kLanes;
      const uint32_t win = group.min_u32(at);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + i * kLanes == (int)win) {
          key[i] = 0;
          s = score[i];
        }
      s = W == 1 ? __shfl_sync(0xffffffffu, s, win % 32) : group.sum_f(s);  // the other lanes hold 0
      sum += s;
      if (lane == k) {
        my_idx = (int)win;
        my_score = s;
      }
    }
    const float m = a.renorm ? (sum > 0.0f ? a.scale / sum : 0.0f) : a.scale;
    if (lane < a.K) {
      a.topk_idx[row * a.K + lane] = my_idx;
      a.topk_w[row * a.K + lane] = my_idx < 0 ? 0.0f : my_score * m;
    }
  }
}

template <int V>
int launch_router_warp(const RouterArgs& a, llmoe_stream_t stream) {
  const int64_t warps = 8, wave = (int64_t)num_sms() * 8;
  const unsigned grid = (unsigned)std::min<int64_t>(wave, (a.rows + warps - 1) / warps);
  return launch_block(router_kernel<1, V>, grid, 256, 0, stream, a);
}

}  // namespace

extern "C" int llmoe_topk_router(const void* logits, const float* bias, const uint8_t* active, int64_t* topk_idx,
                                 float* topk_w, int64_t rows, int num_experts, int num_topk, int dtype, int scoring,
                                 uint32_t flags, float scale, llmoe_stream_t stream) {
  const int es = dtype == LLMOE_DTYPE_FP32 ? 4 : 2;
  if ((dtype != LLMOE_DTYPE_BF16 && dtype != LLMOE_DTYPE_FP16 && dtype != LLMOE_DTYPE_FP32) || num_experts < 1 ||
      num_experts > LLMOE_MAX_EXPERTS || num_topk < 1 || num_topk > LLMOE_MAX_TOPK || num_topk > num_experts ||
      (scoring != LLMOE_SCORE_SIGMOID && scoring != LLMOE_SCORE_SOFTMAX) || (flags & ~LLMOE_ROUTER_RENORM) != 0 ||
      rows < 0 || rows > INT64_MAX / 8 / num_experts)
    return LLMOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return LLMOE_SUCCESS;
  if (logits == nullptr || topk_idx == nullptr || topk_w == nullptr || !aligned(logits, es) || !aligned(bias, 4) ||
      !aligned(topk_idx, 8) || !aligned(topk_w, 4))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const RouterArgs a{logits,      bias,     active, topk_idx, topk_w, rows, num_experts, num_topk,
                     dtype, scoring == LLMOE_SCORE_SOFTMAX, (flags & LLMOE_ROUTER_RENORM) != 0, scale};
  if (num_experts <= 32) return launch_router_warp<1>(a, stream);
  if (num_experts <= 64) return launch_router_warp<2>(a, stream);
  if (num_experts <= 128) return launch_router_warp<4>(a, stream);
  if (num_experts <= 256) return launch_router_warp<8>(a, stream);
  if (num_experts <= 512) return launch_router_warp<16>(a, stream);
  const unsigned grid = (unsigned)std::min<int64_t>((int64_t)num_sms() * 8, rows);
  if (num_experts <= 2048) return launch_block(router_kernel<8, 8>, grid, 256, 0, stream, a);
  return launch_block(router_kernel<8, 32>, grid, 256, 0, stream, a);
}
