// block_group_router.cu -- llmoe_group_router (include/llmoe_block.h).
//
// Where the number of groups divides 32 and a warp's registers hold a row (512
// experts), a warp owns a token and 32 / num_groups lanes a group of experts
// (lanes_kernel): a group's best two keys come from a butterfly over its lanes,
// groups are ranked by counting those ahead of them, and the experts are chosen
// from the few keys that reach a bound: the K-th largest of the kept lanes' best
// keys, which at least K keys do.  Those few go to shared memory, a lane each, and
// their rank among them, counted too, is their place in the result.  Keys are
// 32-bit integers that order like the floats (0: cannot be chosen).
// Instructions bound a large batch: 8192 tokens of 256 experts in 8 groups 7.8 us (with
// keys in shared memory, a lane scoring whole groups and K rounds of reductions over
// all keys 21.3), one token 2.3; 4096 tokens of 160 experts, softmax, 5.4-5.6.  Logits
// of 16 bits are loaded one by one: 8192 x 256 in bf16 10.6.  One expert masked by
// -infinity in every token, so that all take the general reciprocal: 8.6.
// Any other row lies in shared memory as keys (rows_kernel, a warp or, above 512
// experts, a CTA of eight): a lane scores whole groups, and K rounds choose.  8192
// tokens of 160 experts in 5 groups 16.0 us, one 5.3; of 1024 experts in 8 groups 164,
// one 8.6, where 512 take 11.2 and 2.7: a lane reads its group's 128 keys in turn, the
// others wait.
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

// A group's score from its best two keys (second: 0 where there is one, or the score
// is of the best alone), 0 where nothing can be chosen.
__device__ __forceinline__ uint32_t group_score(uint32_t best, uint32_t second) {
  return second == 0 ? best : score_order(unorder(best) + unorder(second));
}

// The row's result from a warp's choices: `place` of lane's expert `mine` (-1: none),
// whose logit is v; places from `chosen` on have none.  top, total: an
// unrenormalised softmax's, over all experts.
template <bool kSoftmax>
__device__ __forceinline__ void store_choice(const GroupRouterArgs& a, int64_t row, int mine, float v, int place,
                                             int chosen, float top, float total) {
  const int lane = threadIdx.x & 31;
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
  if (mine >= 0) {
    a.topk_idx[row * a.K + place] = mine;
    a.topk_w[row * a.K + place] = s * a.scale;
  }
  if (lane >= chosen && lane < a.K) {
    a.topk_idx[row * a.K + lane] = -1;
    a.topk_w[row * a.K + lane] = 0.0f;
  }
}

template <int W, bool kSoftmax>
__global__ void __launch_bounds__(256) rows_kernel(GroupRouterArgs a) {
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
      score[g] = group_score(best, a.top2 ? second : 0);
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
    store_choice<kSoftmax>(a, row, mine, v, lane, __popc(__ballot_sync(0xffffffffu, mine >= 0)), top, total);
  }
}

// order() of a key that is NaN where its logit may not be chosen, and never -0: a sum
// of 1 / (1 + exp(-l)) and a bias (l of -infinity: one_over gives NaN).
__device__ __forceinline__ uint32_t order_of_sum(float key) {
  const uint32_t b = __float_as_uint(key);
  return key > -INFINITY ? b ^ ((uint32_t)((int)b >> 31) | 0x80000000u) : 0u;
}

// V: experts a lane holds at most; kVec: fp32 logits, four experts of a lane in a row.
// Biases are asked for with the logits (read where they are added: 9.1 us against 8.7).
// Experts that a lane has not are NaN: no key, and not far.  A masked token's logits are
// asked for too, not behind its mask (8.1 us against 7.9, a tenth masked).
// CTAs an SM: a softmax keeps its logits too, and with 51 registers a thread, not 64,
// asks for them in parts (6.4 us against 5.4); a large sigmoid gains by a fifth CTA (8.2, 8.1).
template <int V, bool kVec, bool kSoftmax>
__global__ void __launch_bounds__(256, V > 8 ? 3 : kSoftmax ? 4 : 5) lanes_kernel(GroupRouterArgs a) {
  __shared__ __align__(16) uint64_t gathered[8][32];  // a key, and below it ~expert: the lower of equals is ahead
  wait_prior_grid();
  release_next_grid();
  const int lane = threadIdx.x & 31, L = 32 / a.G, g = lane / L, q = lane - g * L;
  uint64_t* list = gathered[threadIdx.x >> 5];
  // the lane's i-th expert, of its group: in order over the group's lanes, or four in a row
  const auto expert = [&](int i) { return kVec ? (i / 4 * L + q) * 4 + i % 4 : i * L + q; };
  const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; row < a.rows; row += step) {
    const bool on = a.active == nullptr || a.active[row] != 0;
    const int64_t at = row * a.E + g * a.S;
    float l[V], b[V];
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.bias != nullptr && expert(i) < a.S) v = *reinterpret_cast<const float4*>(a.bias + g * a.S + expert(i));
        b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = a.bias != nullptr && expert(i) < a.S ? a.bias[g * a.S + expert(i)] : 0.0f;
    }
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        float4 v = make_float4(NAN, NAN, NAN, NAN);
        if (expert(i) < a.S) v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at + expert(i));
        l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = expert(i) < a.S ? load_logit(a.logits, a.dtype, at + expert(i)) : NAN;
    }
    if (!on) {  // chooses nothing
      if (lane < a.K) a.topk_idx[row * a.K + lane] = -1, a.topk_w[row * a.K + lane] = 0.0f;
      continue;
    }
    uint32_t key[V], best = 0, second = 0;
    const auto keys = [&](auto score, auto order) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float k = score(l[i]);
        k += b[i];
        key[i] = order(l[i], k);
        second = max(second, min(best, key[i]));
        best = max(best, key[i]);
      }
    };
    if constexpr (kSoftmax) {
      keys([](float v) { return v; }, order);
    } else {
      float far = 0.0f;  // NaN is not far
#pragma unroll
      for (int i = 0; i < V; ++i) far = fmaxf(far, -l[i]);
      if (__all_sync(0xffffffffu, far <= 87.0f))
        keys([](float v) { return one_over(1.0f + expf(-v)); }, [](float, float k) { return order_of_sum(k); });
      else
        keys([](float v) { return sigmoid_score(v); }, order);
    }
    float top = -INFINITY, total = 0.0f;
    if (kSoftmax && !a.renorm) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] != 0) top = fmaxf(top, l[i]);
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] != 0) total += softmax_score(l[i], top);
#pragma unroll
      for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    }
    uint32_t lane_best = best;
    if (a.kept < a.G) {
      if (a.top2) {
        for (int d = 1; d < L; d <<= 1) {
          const uint32_t b = __shfl_xor_sync(0xffffffffu, best, d), s = __shfl_xor_sync(0xffffffffu, second, d);
          second = max(max(second, s), min(best, b));
          best = max(best, b);
        }
      } else {
        second = 0;
        for (int d = 1; d < L; d <<= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
      }
      const uint32_t score = group_score(best, second);
      int ahead = 0;  // the group's lanes count a part of the others each (all by each: 8.3 us against 8.2)
#pragma unroll 1
      for (int first = 0; first < a.G; first += L) {
        const int o = first + q;
        const uint32_t other = __shfl_sync(0xffffffffu, score, o * L);
        ahead += o < a.G && (other > score || (other == score && o < g));
      }
      for (int d = 1; d < L; d <<= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, d);
      if (ahead >= a.kept) {
        lane_best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 0;
      }
    }
    uint32_t bound = 0, left = lane_best;
    for (int k = 0; k < a.K; ++k) {
      bound = __reduce_max_sync(0xffffffffu, left);
      if (left == bound) left = 0;
    }
    const uint32_t least = max(bound, 1u);
    int n = 0;
    __syncwarp();  // the previous row's list has been read
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = key[i] >= least;
      const uint32_t who = __ballot_sync(0xffffffffu, in);
      const int to = n + __popc(who & ((1u << lane) - 1));
      if (in && to < 32) list[to] = (uint64_t)key[i] << 32 | (uint32_t)~(g * a.S + expert(i));
      n += __popc(who);
    }
    __syncwarp();
    if (n <= 32) {
      if (lane >= n) list[lane] = 0;
      __syncwarp();
      const uint64_t mine = list[lane];
      const int e = (int)~(uint32_t)mine;
      int place = 0;
      for (int o = 0; o < n; o += 4) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(list + o), y = *reinterpret_cast<const ulonglong2*>(list + o + 2);
        place += (x.x > mine) + (x.y > mine) + (y.x > mine) + (y.y > mine);
      }
      const bool chosen = lane < n && place < a.K;
      const float v = chosen ? load_logit(a.logits, a.dtype, row * a.E + e) : -INFINITY;
      store_choice<kSoftmax>(a, row, chosen ? e : -1, v, place, min(n, a.K), top, total);
      continue;
    }
    // many keys at the bound, or few lanes: rounds of two reductions, over all keys
    int mine = -1;
    float v = -INFINITY;
    for (int k = 0; k < a.K; ++k) {
      uint32_t most = 0, e = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t at_e = (uint32_t)(g * a.S + expert(i));
        if (key[i] > most || (key[i] == most && most != 0 && at_e < e)) most = key[i], e = at_e;
      }
      const uint32_t win = __reduce_max_sync(0xffffffffu, most);
      if (win == 0) break;
      e = __reduce_min_sync(0xffffffffu, most == win ? e : 0xffffffffu);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] != 0 && (uint32_t)(g * a.S + expert(i)) == e) key[i] = 0;
      if (lane == k) mine = (int)e;
    }
    if (mine >= 0) v = load_logit(a.logits, a.dtype, row * a.E + mine);
    store_choice<kSoftmax>(a, row, mine, v, lane, __popc(__ballot_sync(0xffffffffu, mine >= 0)), top, total);
  }
}

template <int V, bool kSoftmax>
int launch_lanes(const GroupRouterArgs& a, bool vec, llmoe_stream_t stream) {
  const unsigned grid = (unsigned)std::min<int64_t>((int64_t)num_sms() * 8, (a.rows + 7) / 8);
  if constexpr (V >= 4)
    if (vec) return launch_block(lanes_kernel<V, true, kSoftmax>, grid, 256, 0, stream, a);
  return launch_block(lanes_kernel<V, false, kSoftmax>, grid, 256, 0, stream, a);
}

template <bool kSoftmax>
int launch_group_router(const GroupRouterArgs& a, llmoe_stream_t stream) {
  if (32 % a.G == 0) {
    const int L = 32 / a.G, each = (a.S + L - 1) / L;  // experts a lane holds
    // a lane's experts four in a row where the group's are whole fours for each lane
    const bool vec = a.dtype == LLMOE_DTYPE_FP32 && a.S % (4 * L) == 0 && aligned(a.logits, 16) && aligned(a.bias, 16);
    if (each <= 1) return launch_lanes<1, kSoftmax>(a, vec, stream);
    if (each <= 2) return launch_lanes<2, kSoftmax>(a, vec, stream);
    if (each <= 4) return launch_lanes<4, kSoftmax>(a, vec, stream);
    if (each <= 8) return launch_lanes<8, kSoftmax>(a, vec, stream);
    if (each <= 16) return launch_lanes<16, kSoftmax>(a, vec, stream);
  }
  const size_t words = (size_t)a.E + a.G;
  if (a.E <= 512) {
    const unsigned grid = (unsigned)std::min<int64_t>((int64_t)num_sms() * 8, (a.rows + 7) / 8);
    return launch_block(rows_kernel<1, kSoftmax>, grid, 256, 8 * words * 4, stream, a);
  }
  const unsigned grid = (unsigned)std::min<int64_t>((int64_t)num_sms() * 4, a.rows);
  return launch_block(rows_kernel<8, kSoftmax>, grid, 256, words * 4, stream, a);
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
