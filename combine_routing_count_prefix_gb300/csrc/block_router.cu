// block_router.cu -- llmoe_topk_router (include/llmoe_block.h).
//
// A group of one warp (a CTA of eight for more experts than a warp holds in
// registers) owns a token; a lane holds its experts' keys as 32-bit integers
// that order like the floats (0: cannot be chosen).  The choice is K rounds of
// two warp reductions, the largest key and, among its holders, the lowest
// expert, so ties go to the lowest index whatever the schedule.
//
// Bytes are few (1 KB a token); what bounds a large batch is the instructions
// issued.  So a warp first finds the few experts that can be chosen at all: the
// K-th largest of the 32 lanes' best keys is a bound that at least K keys reach
// (K = 8 of 256: about ten do), and for that keys from the hardware's
// exponential and reciprocal are enough, with a margin for their error.  Those
// few go one to a lane, which computes their fp32 keys as defined, and the
// rounds run over them.  8192 tokens of 256 experts, sigmoid: 8.6 us with exact
// keys for all, 7.7 with this; 7.3 with a kernel for each scoring (a softmax 7.2
// renormalised, 7.8 not), one token 3.0.  About 710 instructions a token.
#include <float.h>

#include "block_router.cuh"

namespace {

struct RouterArgs {
  const void* logits;
  const float* bias;
  const uint8_t* active;
  int64_t* topk_idx;
  float* topk_w;
  int64_t rows;
  int E, K, dtype;
  bool renorm;
  float scale;
};

// The expert that lane `lane` of a group holds as its i-th: in order over the
// lanes, or (kVec) four in a row, so that they load as one.
template <int W, bool kVec>
__device__ __forceinline__ int expert_of(int lane, int i) {
  constexpr int kLanes = 32 * W;
  return kVec ? (i / 4 * kLanes + lane) * 4 + i % 4 : lane + i * kLanes;
}

template <bool kSoftmax>
__device__ __forceinline__ uint32_t exact_key(const RouterArgs& a, int e, float l) {
  float k = kSoftmax ? l : sigmoid_score(l);
  if (a.bias != nullptr) k += a.bias[e];
  return order(l, k);
}

// W warps per token, V experts per lane; kVec: fp32 logits, rows of whole 16
// bytes.  A kernel for each scoring: in one for both, what the softmax keeps of
// an expert's key cost the sigmoid 3 to 6% of 8192 tokens of 256 experts.
template <int W, int V, bool kVec, bool kSoftmax>
__global__ void __launch_bounds__(256, W > 1 || V > 8 ? 2 : 5) router_kernel(RouterArgs a) {
  __shared__ uint32_t part[W];
  __shared__ uint2 gathered[W == 1 ? 8 : 1][32];
  wait_prior_grid();
  release_next_grid();
  const Group<W> group{part};
  const int lane = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t first = W == 1 ? ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5 : blockIdx.x;
  const int64_t step = W == 1 ? ((int64_t)gridDim.x * blockDim.x) >> 5 : gridDim.x;
  for (int64_t row = first; row < a.rows; row += step) {
    const bool on = a.active == nullptr || a.active[row] != 0;
    float l[V];
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int e = expert_of<W, kVec>(lane, i);
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (on && e < a.E) q = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + row * a.E + e);
        l[i] = q.x, l[i + 1] = q.y, l[i + 2] = q.z, l[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = expert_of<W, kVec>(lane, i);
        l[i] = on && e < a.E ? load_logit(a.logits, a.dtype, row * a.E + e) : -INFINITY;
      }
    }
    constexpr bool kFew = W == 1 && V > 1;
    float near[V];    // kFew: keys by hardware arithmetic (a softmax's are exact)
    uint32_t key[V];  // otherwise, and where near keys leave too many: the exact ones' order
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert_of<W, kVec>(lane, i);
      if constexpr (kFew) {
        near[i] = kSoftmax ? l[i] : __fdividef(1.0f, 1.0f + __expf(-l[i]));
        if (a.bias != nullptr && e < a.E) near[i] += a.bias[e];
        if (kSoftmax && !(near[i] > -INFINITY)) l[i] = -INFINITY;  // an expert that the bias masks is none of the softmax's
        if (!(l[i] > -INFINITY)) near[i] = -INFINITY;
      } else {
        key[i] = e < a.E ? exact_key<kSoftmax>(a, e, l[i]) : 0u;
        if (kSoftmax && key[i] == 0u) l[i] = -INFINITY;
      }
    }
    float top = -INFINITY, total = 0.0f;
    if (kSoftmax && !a.renorm) {
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
      top = group.max_f(top);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (l[i] > -INFINITY) total += softmax_score(l[i], top);
      total = group.sum_f(total);
    }

    int mine = -1;  // lane k of the first warp keeps the k-th choice
    bool rounds = true;
    if constexpr (kFew) {
      float left = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) left = fmaxf(left, near[i]);
      uint32_t lane_best = order(left, left), bound = 0;
      for (int k = 0; k < a.K; ++k) {
        bound = group.max_u32(lane_best);
        if (bound == 0) break;
        if (lane_best == bound) lane_best = 0;
      }
      // |near - key| <= 2^-20 + 2^-23 |key|: the exponential is within (2 + 1.2 |l|)
      // ulp, which s (1 - s) damps, the division within 2 ulp, the sums round.  A
      // chosen key is at most that below the bound, its near value twice that.
      float least = -FLT_MAX;
      if (bound != 0) {
        const float b = unorder(bound);
        least = b == INFINITY || kSoftmax ? b : b - (0x1p-18f + fabsf(b) * 0x1p-21f);
      }
      uint2* list = gathered[threadIdx.x >> 5];
      int n = 0;
      __syncwarp();  // the previous row's list has been read
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool in = near[i] >= least;
        const uint32_t who = __ballot_sync(0xffffffffu, in);
        const int at = n + __popc(who & ((1u << lane) - 1));
        if (in && at < 32) list[at] = make_uint2(__float_as_uint(l[i]), (uint32_t)expert_of<W, kVec>(lane, i));
        n += __popc(who);
      }
      __syncwarp();
      if (n <= 32) {
        rounds = false;
        const uint2 q = lane < n ? list[lane] : make_uint2(0, 0);
        uint32_t best = lane < n ? exact_key<kSoftmax>(a, (int)q.y, __uint_as_float(q.x)) : 0u;
        for (int k = 0; k < a.K; ++k) {
          const uint32_t win = group.max_u32(best);
          if (win == 0) break;
          const int e = (int)group.min_u32(best == win ? q.y : 0xffffffffu);
          if (best == win && (int)q.y == e) best = 0;
          if (lane == k) mine = e;
        }
      }
    }
    if (rounds) {  // over all keys: many equal ones at the bound, or a CTA per token
      if constexpr (kFew) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = expert_of<W, kVec>(lane, i);
          key[i] = e < a.E ? exact_key<kSoftmax>(a, e, l[i]) : 0u;
        }
      }
      uint32_t best;  // this lane's largest key left, and its expert
      int best_e;
      const auto look = [&] {
        best = 0, best_e = INT_MAX;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i] > best) best = key[i], best_e = expert_of<W, kVec>(lane, i);
      };
      look();
      for (int k = 0; k < a.K; ++k) {
        const uint32_t win = group.max_u32(best);
        if (win == 0) break;  // nothing left to choose: uniform over the group
        const int e = (int)group.min_u32(best == win ? (uint32_t)best_e : 0xffffffffu);
        if (best == win && best_e == e) {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (expert_of<W, kVec>(lane, i) == e) key[i] = 0;
          look();
        }
        if (lane == k) mine = e;
      }
    }
    if (W > 1 && lane >= 32) continue;
    const float v = mine >= 0 ? load_logit(a.logits, a.dtype, row * a.E + mine) : -INFINITY;
    if (kSoftmax && a.renorm) {
      // what is renormalised is a softmax of the chosen alone: relative to the
      // largest of them, which the row's largest may be above by more than an
      // fp32 score can be small
      top = v;
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    float score = 0.0f;
    if (mine >= 0) score = !kSoftmax ? sigmoid_score(v) : a.renorm ? softmax_score(v, top) : softmax_score(v, top) / total;
    if (a.renorm) {
      float sum = score;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      score = sum > 0.0f ? score / sum : 0.0f;  // before the scale: scale / sum may be above fp32's largest
    }
    if (lane < a.K) {
      a.topk_idx[row * a.K + lane] = mine;
      a.topk_w[row * a.K + lane] = score * a.scale;
    }
  }
}

// Experts per lane: a power of two, so that a few kernels serve all E.
template <int V, bool kSoftmax>
int launch_router_warp(const RouterArgs& a, bool vec, llmoe_stream_t stream) {
  const int64_t warps = 8, wave = (int64_t)num_sms() * 8;
  const unsigned grid = (unsigned)std::min<int64_t>(wave, (a.rows + warps - 1) / warps);
  if constexpr (V >= 4)
    if (vec) return launch_block(router_kernel<1, V, true, kSoftmax>, grid, 256, 0, stream, a);
  return launch_block(router_kernel<1, V, false, kSoftmax>, grid, 256, 0, stream, a);
}

template <bool kSoftmax>
int launch_router(const RouterArgs& a, bool vec, llmoe_stream_t stream) {
  if (a.E <= 32) return launch_router_warp<1, kSoftmax>(a, vec, stream);
  if (a.E <= 64) return launch_router_warp<2, kSoftmax>(a, vec, stream);
  if (a.E <= 128) return launch_router_warp<4, kSoftmax>(a, vec, stream);
  if (a.E <= 256) return launch_router_warp<8, kSoftmax>(a, vec, stream);
  if (a.E <= 512) return launch_router_warp<16, kSoftmax>(a, vec, stream);
  const unsigned grid = (unsigned)std::min<int64_t>((int64_t)num_sms() * 8, a.rows);
  if (a.E <= 2048) return launch_block(router_kernel<8, 8, false, kSoftmax>, grid, 256, 0, stream, a);
  return launch_block(router_kernel<8, 32, false, kSoftmax>, grid, 256, 0, stream, a);
}

}  // namespace

extern "C" int llmoe_topk_router(const void* logits, const float* bias, const uint8_t* active, int64_t* topk_idx,
                                 float* topk_w, int64_t rows, int num_experts, int num_topk, int dtype, int scoring,
                                 uint32_t flags, float scale, llmoe_stream_t stream) {
  if (!router_shape(rows, num_experts, num_topk, dtype, scoring) || (flags & ~LLMOE_ROUTER_RENORM) != 0)
    return LLMOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return LLMOE_SUCCESS;
  if (!router_memory(logits, bias, active, topk_idx, topk_w, rows, num_experts, num_topk, dtype))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const RouterArgs a{logits,      bias,     active, topk_idx, topk_w, rows, num_experts, num_topk,
                     dtype, (flags & LLMOE_ROUTER_RENORM) != 0, scale};
  const bool vec = dtype == LLMOE_DTYPE_FP32 && num_experts % 4 == 0 && aligned(logits, 16);
  return scoring == LLMOE_SCORE_SOFTMAX ? launch_router<true>(a, vec, stream) : launch_router<false>(a, vec, stream);
}
