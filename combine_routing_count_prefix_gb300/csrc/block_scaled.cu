// block_scaled.cu -- llmoe_expert_product_fp8b (include/llmoe_block.h).
//
// A thread holds one feature of one received row: a CTA takes 128 features and
// two slots of a bucket at a time.
#include "block_plan.cuh"

namespace {

struct ScaledArgs {
  ProductArgs p;
  const float* w_scale;
  int down, across;  // blocks of 128 down and across one matrix of w
};

__device__ __forceinline__ float e4m3(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <bool kSwiglu>
__global__ void __launch_bounds__(256) scaled_kernel(ScaledArgs s) {
  constexpr int kParts = kSwiglu ? 2 : 1;
  __shared__ uint32_t most[2][4];
  wait_prior_grid();
  release_next_grid();
  const ProductArgs& a = s.p;
  const int tid = threadIdx.x, tiles = (a.out + 127) / 128;
  const int64_t jobs = (int64_t)a.E * a.R * tiles;
  for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int tile = (int)(job % tiles), bucket = (int)(job / tiles), e = bucket / a.R;
    int count[1];
    bucket_counts(a, e, bucket % a.R, a.R, count);
    const int f = tile * 128 + (tid & 127);
    const bool in = f < a.out;
    for (int slot = tid >> 7; slot < (count[0] + 1) / 2 * 2; slot += 2) {
      const int64_t row = (int64_t)bucket * a.T + min(slot, count[0] - 1);
      const uint8_t* x = a.x + row * a.x_row;
      const float* xs = reinterpret_cast<const float*>(x + a.in);
      float sum[kParts] = {};
      for (int b = 0; b < a.steps; ++b) {
        const int k1 = min(a.in, 128 * (b + 1));
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          const uint8_t* w = a.w + (((uint64_t)e * kParts + p) * a.out + min(f, a.out - 1)) * a.in;
          float part = 0.0f;
          for (int k = 128 * b; k < k1; ++k) part += e4m3(x[k]) * e4m3(w[k]);
          const float ws = s.w_scale[(((int64_t)e * kParts + p) * s.down + tile) * s.across + b];
          sum[p] = fmaf(part, xs[b] * ws, sum[p]);
        }
      }
      float v = kSwiglu ? silu(sum[0]) * sum[kParts - 1] : sum[0];
      uint8_t* y = a.y + row * a.y_row;
      const bool store = in && slot < count[0];
      if (a.out_dtype == LLMOE_DTYPE_FP8B) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, in ? magnitude(v) : 0u);
        __syncthreads();
        if ((tid & 31) == 0) most[tid >> 7][tid >> 5 & 3] = m;
        __syncthreads();
        uint32_t amax = 0;
        for (int i = 0; i < 4; ++i) amax = max(amax, most[tid >> 7][i]);
        const float scale = block_scale(__uint_as_float(amax));
        if (store) {
          y[f] = (uint8_t)pack_e4m3x2(v * __frcp_rn(scale), 0.0f);
          if ((tid & 127) == 0) reinterpret_cast<float*>(y + a.out)[tile] = scale;
          if (f == a.out - 1)
            for (uint32_t i = a.out + tiles * 4; i < a.y_row; ++i) y[i] = 0;
        }
      } else if (store) {
        if (a.out_dtype == LLMOE_DTYPE_FP32)
          reinterpret_cast<float*>(y)[f] = v;
        else if (a.out_dtype == LLMOE_DTYPE_FP16)
          reinterpret_cast<__half*>(y)[f] = __float2half_rn(v);
        else
          reinterpret_cast<__nv_bfloat16*>(y)[f] = __float2bfloat16_rn(v);
      }
    }
  }
}

int launch_scaled(const ScaledArgs& s, bool swiglu, llmoe_stream_t stream) {
  const int64_t jobs = (int64_t)s.p.E * s.p.R * ((s.p.out + 127) / 128);
  const unsigned grid = (unsigned)std::min<int64_t>(jobs, (int64_t)num_sms() * 8);
  return swiglu ? launch_block(scaled_kernel<true>, grid, 256, 0, stream, s)
                : launch_block(scaled_kernel<false>, grid, 256, 0, stream, s);
}

}  // namespace

extern "C" int llmoe_expert_product_fp8b(const void* x, const void* w, const float* w_scale, void* y,
                                         const int64_t* counts, int in_features, int out_features, int out_dtype,
                                         uint32_t flags, const llmoe_buf_set_t* bs, llmoe_stream_t stream) {
  ScaledArgs s;
  ProductArgs& a = s.p;
  const bool swiglu = (flags & LLMOE_PRODUCT_SWIGLU) != 0;
  if ((flags & ~LLMOE_PRODUCT_SWIGLU) != 0 || !product_buckets(counts, bs, &a) ||
      !(out_dtype == LLMOE_DTYPE_BF16 || out_dtype == LLMOE_DTYPE_FP16 || out_dtype == LLMOE_DTYPE_FP32 ||
        (out_dtype == LLMOE_DTYPE_FP8B && swiglu)) ||
      !product_rows(x, y, in_features, out_features, LLMOE_DTYPE_FP8B, out_dtype, swiglu, &a))
    return LLMOE_ERR_INVALID_ARGUMENT;
  s.down = (out_features + LLMOE_FP8B_BLOCK - 1) / LLMOE_FP8B_BLOCK;
  s.across = (int)(((int64_t)in_features + LLMOE_FP8B_BLOCK - 1) / LLMOE_FP8B_BLOCK);
  const uint64_t matrices = (uint64_t)a.E * (swiglu ? 2 : 1), codes = (uint64_t)out_features * in_features;
  if (w == nullptr || w_scale == nullptr || !aligned(w, 16) || !aligned(w_scale, 4) || codes > kMostBytes / matrices)
    return LLMOE_ERR_INVALID_ARGUMENT;
  const uint64_t y_bytes = (uint64_t)a.E * a.R * a.T * a.y_row;
  if (overlap(y, y_bytes, w, matrices * codes) || overlap(y, y_bytes, w_scale, matrices * s.down * s.across * 4))
    return LLMOE_ERR_INVALID_ARGUMENT;
  a.w = static_cast<const uint8_t*>(w);
  s.w_scale = w_scale;
  a.steps = s.across;
  return launch_scaled(s, swiglu, stream);
}
