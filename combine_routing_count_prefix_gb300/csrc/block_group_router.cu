// block_group_router.cu -- llmoe_group_router (include/llmoe_block.h).
//
// A group of one warp (a CTA of eight for many experts) owns a token.  Its keys,
// 32-bit integers that order like the floats (0: cannot be chosen), lie in shared
// memory; a lane finds the score of whole groups of experts, groups are ranked by
// counting those ahead of them, and K rounds of two reductions choose the experts.
#include "block_router.cuh"

namespace {

struct GroupRouterArgs {
  const void* logits;
  const float* bias;
  const uint8_t* active;
  int64_t* topk_idx;
  float* topk_w;
  int64_t rows;
  int E, K, G, S, kept, dtype;  // S: experts per group
  bool renorm, top2;
  float scale;
};

template <int W>
__device__ __forceinline__ void group_sync() {
  if constexpr (W == 1)
    __syncwarp();
  else
    __syncthreads();
}

// A group's score as an integer of the same order, above 0.
__device__ __forceinline__ uint32_t score_order(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <int W, bool kSoftmax>
__global__ void __launch_bounds__(256) group_router_kernel(GroupRouterArgs a) {
  extern __shared__ uint32_t smem[];
  __shared__ uint32_t part[W];
  wait_prior_grid();
  release_next_grid();
  constexpr int kLanes = 32 * W;
  const Group<W> group{part};
  const int lane = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  uint32_t* key = smem + (W == 1 ? (threadIdx.x >> 5) * (a.E + a.G) : 0);
  uint32_t* score = key + a.E;
  const int64_t first = W == 1 ? ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5 : blockIdx.x;
  const int64_t step = W == 1 ? ((int64_t)gridDim.x * blockDim.x) >> 5 : gridDim.x;
  for (int64_t row = first; row < a.rows; row += step) {
    const bool on = a.active == nullptr || a.active[row] != 0;
    group_sync<W>();  // the previous row's keys have been read
    float top = -INFINITY, total = 0.0f;
    for (int e = lane; e < a.E; e += kLanes) {
      const float l = on ? load_logit(a.logits, a.dtype, row * a.E + e) : -INFINITY;
      float k = kSoftmax ? l : sigmoid_score(l);
      if (a.bias != nullptr) k += a.bias[e];
      key[e] = order(l, k);
      if (key[e] != 0) top = fmaxf(top, l);
    }
    if (kSoftmax && !a.renorm) {
      top = group.max_f(top);
      for (int e = lane; e < a.E; e += kLanes)
        if (key[e] != 0) total += softmax_score(load_logit(a.logits, a.dtype, row * a.E + e), top);
      total = group.sum_f(total);
    }
    group_sync<W>();
    for (int g = lane; g < a.G; g += kLanes) {
      uint32_t best = 0, second = 0;
      for (int i = 0; i < a.S; ++i) {
        const uint32_t k = key[g * a.S + i];
        second = max(second, min(best, k));
        best = max(best, k);
      }
      score[g] = best == 0 ? 0 : a.top2 && second != 0 ? score_order(unorder(best) + unorder(second)) : best;
    }
    group_sync<W>();
    for (int g = lane; g < a.G; g += kLanes) {
      const uint32_t mine = score[g];
      int ahead = 0;
      for (int o = 0; o < a.G; ++o) ahead += score[o] > mine || (score[o] == mine && o < g);
      if (ahead >= a.kept)
        for (int i = 0; i < a.S; ++i) key[g * a.S + i] = 0;
    }
    group_sync<W>();
    int mine = -1;  // lane k of the first warp keeps the k-th choice
    for (int k = 0; k < a.K; ++k) {
      uint32_t best = 0;
      int best_e = INT_MAX;
      for (int e = lane; e < a.E; e += kLanes)
        if (key[e] > best) best = key[e], best_e = e;
      const uint32_t win = group.max_u32(best);
      if (win == 0) break;  // nothing left to choose: uniform over the group
      const int e = (int)group.min_u32(best == win ? (uint32_t)best_e : 0xffffffffu);
      if (best_e == e) key[e] = 0;
      if (lane == k) mine = e;
    }
    if (W > 1 && lane >= 32) continue;
    const float v = mine >= 0 ? load_logit(a.logits, a.dtype, row * a.E + mine) : -INFINITY;
    if (kSoftmax && a.renorm) {  // a softmax of the chosen alone
      top = v;
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    float s = 0.0f;
    if (mine >= 0) s = !kSoftmax ? sigmoid_score(v) : a.renorm ? softmax_score(v, top) : softmax_score(v, top) / total;
    if (a.renorm) {
      float sum = s;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      s = sum > 0.0f ? s / sum : 0.0f;  // before the scale: scale / sum may be above fp32's largest
    }
    if (lane < a.K) {
      a.topk_idx[row * a.K + lane] = mine;
      a.topk_w[row * a.K + lane] = s * a.scale;
    }
  }
}

template <bool kSoftmax>
int launch_group_router(const GroupRouterArgs& a, llmoe_stream_t stream) {
  const size_t words = (size_t)a.E + a.G;
  if (a.E <= 512) {
    const unsigned grid = (unsigned)std::min<int64_t>((int64_t)num_sms() * 8, (a.rows + 7) / 8);
    return launch_block(group_router_kernel<1, kSoftmax>, grid, 256, 8 * words * 4, stream, a);
  }
  const unsigned grid = (unsigned)std::min<int64_t>((int64_t)num_sms() * 4, a.rows);
  return launch_block(group_router_kernel<8, kSoftmax>, grid, 256, words * 4, stream, a);
}

}  // namespace

extern "C" int llmoe_group_router(const void* logits, const float* bias, const uint8_t* active, int64_t* topk_idx,
                                  float* topk_w, int64_t rows, int num_experts, int num_topk, int num_groups,
                                  int kept_groups, int dtype, int scoring, uint32_t flags, float scale,
                                  llmoe_stream_t stream) {
  if (!router_shape(rows, num_experts, num_topk, dtype, scoring) ||
      (flags & ~(LLMOE_ROUTER_RENORM | LLMOE_ROUTER_GROUP_TOP2)) != 0 || num_groups < 1 ||
      num_groups > LLMOE_MAX_GROUPS || num_experts % num_groups != 0 || kept_groups < 1 || kept_groups > num_groups ||
      num_topk > num_experts / num_groups * kept_groups ||
      ((flags & LLMOE_ROUTER_GROUP_TOP2) != 0 && scoring != LLMOE_SCORE_SIGMOID))
    return LLMOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return LLMOE_SUCCESS;
  if (!router_memory(logits, bias, active, topk_idx, topk_w, rows, num_experts, num_topk, dtype))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const GroupRouterArgs a{logits, bias, active, topk_idx, topk_w, rows, num_experts, num_topk, num_groups,
                          num_experts / num_groups, kept_groups, dtype, (flags & LLMOE_ROUTER_RENORM) != 0,
                          (flags & LLMOE_ROUTER_GROUP_TOP2) != 0, scale};
  return scoring == LLMOE_SCORE_SOFTMAX ? launch_group_router<true>(a, stream) : launch_group_router<false>(a, stream);
}
