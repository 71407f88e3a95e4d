// block_product.cu -- llmoe_expert_product (include/llmoe_block.h): matrix
// products grouped by expert over the received rows.
//
// Simple form: one CTA per (expert, 64 output features) walks the expert's
// received rows 64 at a time; x and w tiles go through shared memory as fp32
// and every thread accumulates 4 x 4 sums (two sets for gate and up).
#include "block_common.cuh"

namespace {

constexpr int kTile = 64, kStep = 32;

struct ProductArgs {
  const uint8_t* x;
  const uint8_t* w;
  uint8_t* y;
  const int64_t* counts;  // [E][R], or null: the signal words
  const uint8_t* base;    // rank buffers' signal words: base + (e / L) * rank_stride + sig_off
  uint64_t rank_stride, sig_off;
  int32_t* err;
  int T, R, E, L;
  int in, out, n;  // n: rows of w per expert
  uint64_t x_row, y_row;  // bytes
  int dtype, out_dtype;
};

__device__ __forceinline__ int bucket_count(const ProductArgs& a, int e, int src) {
  const int64_t* p = a.counts != nullptr
                         ? a.counts + (int64_t)e * a.R + src
                         : reinterpret_cast<const int64_t*>(a.base + (e / a.L) * a.rank_stride + a.sig_off) +
                               ((int64_t)(e % a.L) * a.R + src);
  const int64_t c = *p;
  if (c < 0 || c > a.T) report(a.err, LLMOE_DEV_SLOT_RANGE);
  return (int)max((int64_t)0, min(c, (int64_t)a.T));
}

__device__ __forceinline__ float load_value(const uint8_t* row, int i, int n, int dtype) {
  switch (dtype) {
    case LLMOE_DTYPE_BF16: return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[i]);
    case LLMOE_DTYPE_FP16: return __half2float(reinterpret_cast<const __half*>(row)[i]);
    default: {
      const uint32_t s = row[n + i / 32];
      const float scale = s == 255 ? __uint_as_float(0x7fffffffu) : s == 0 ? 0x1p-127f : __uint_as_float(s << 23);
      return float(reinterpret_cast<const __nv_fp8_e4m3*>(row)[i]) * scale;
    }
  }
}

template <bool kSwiglu>
__global__ void __launch_bounds__(256) product_kernel(ProductArgs a) {
  __shared__ float xs[kStep][kTile + 1], ws[kSwiglu ? 2 : 1][kStep][kTile + 1];
  __shared__ int64_t rows[kTile];
  __shared__ float os[kTile][kTile + 1];
  release_next_grid();
  wait_prior_grid();
  const int tiles = (a.out + kTile - 1) / kTile;
  const int e = blockIdx.x / tiles, n0 = (blockIdx.x % tiles) * kTile;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const uint8_t* w = a.w + (uint64_t)e * a.n * a.x_row;
  int src = 0, slot = 0;  // thread 0 walks the buckets
  for (;;) {
    __shared__ int s_have;
    if (tid == 0) {
      int have = 0;
      while (have < kTile && src < a.R) {
        if (slot >= bucket_count(a, e, src)) {
          ++src;
          slot = 0;
          continue;
        }
        rows[have++] = ((int64_t)e * a.R + src) * a.T + slot++;
      }
      s_have = have;
    }
    __syncthreads();
    const int have = s_have;
    if (have == 0) return;
    float acc[kSwiglu ? 2 : 1][4][4] = {};
    for (int k0 = 0; k0 < a.in; k0 += kStep) {
      for (int i = tid; i < kTile * kStep; i += 256) {
        const int r = i / kStep, k = i % kStep;
        xs[k][r] = r < have && k0 + k < a.in ? load_value(a.x + rows[r] * a.x_row, k0 + k, a.in, a.dtype) : 0.0f;
#pragma unroll
        for (int h = 0; h < (kSwiglu ? 2 : 1); ++h)
          ws[h][k][r] = n0 + r < a.out && k0 + k < a.in
                            ? load_value(w + ((uint64_t)h * a.out + n0 + r) * a.x_row, k0 + k, a.in, a.dtype)
                            : 0.0f;
      }
      __syncthreads();
      for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int h = 0; h < (kSwiglu ? 2 : 1); ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[h][i][j] += xs[k][ty + 16 * i] * ws[h][k][tx + 16 * j];
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v = acc[0][i][j];
        if constexpr (kSwiglu) v = v / (1.0f + expf(-v)) * acc[1][i][j];
        os[ty + 16 * i][tx + 16 * j] = v;
      }
    __syncthreads();
    if (a.out_dtype == LLMOE_DTYPE_MX8) {
      for (int i = tid; i < have * 2; i += 256) {
        const int r = i / 2, n = n0 + i % 2 * 32;
        if (n >= a.out) continue;
        uint8_t* row = a.y + rows[r] * a.y_row;
        uint32_t amax = 0;
        for (int k = 0; k < 32; ++k) amax = max(amax, magnitude(os[r][n - n0 + k]));
        const uint32_t code = scale_code(amax);
        const float inv = scale_inverse(code);
        for (int k = 0; k < 32; k += 2)
          *reinterpret_cast<uint16_t*>(row + n + k) =
              (uint16_t)pack_e4m3x2(os[r][n - n0 + k] * inv, os[r][n - n0 + k + 1] * inv);
        row[a.out + n / 32] = (uint8_t)code;
        if (n + 32 == a.out)
          for (uint64_t p = a.out + a.out / 32; p < a.y_row; ++p) row[p] = 0;
      }
    } else {
      for (int i = tid; i < have * kTile; i += 256) {
        const int r = i / kTile, n = n0 + i % kTile;
        if (n >= a.out) continue;
        uint8_t* row = a.y + rows[r] * a.y_row;
        const float v = os[r][i % kTile];
        if (a.out_dtype == LLMOE_DTYPE_BF16)
          reinterpret_cast<__nv_bfloat16*>(row)[n] = __float2bfloat16_rn(v);
        else if (a.out_dtype == LLMOE_DTYPE_FP16)
          reinterpret_cast<__half*>(row)[n] = __float2half_rn(v);
        else
          reinterpret_cast<float*>(row)[n] = v;
      }
    }
    __syncthreads();
  }
}

// Checks a product's arguments and fills its geometry.
int product_args(const void* x, const void* w, void* y, const int64_t* counts, int in, int out, int dtype,
                 int out_dtype, uint32_t flags, const llmoe_buf_set_t* bs, ProductArgs* a) {
  if (bs == nullptr || (flags & ~LLMOE_PRODUCT_SWIGLU) != 0) return LLMOE_ERR_INVALID_ARGUMENT;
  const bool swiglu = (flags & LLMOE_PRODUCT_SWIGLU) != 0;
  const int T = bs->num_max_tokens, R = bs->num_ranks, E = bs->num_experts;
  if (T < 1 || R < 1 || E < R || E % R != 0 || E > LLMOE_MAX_EXPERTS || !aligned(bs->err, 4))
    return LLMOE_ERR_INVALID_ARGUMENT;
  if ((uint64_t)E * R > INT32_MAX || (uint64_t)E * R * T > INT32_MAX) return LLMOE_ERR_INVALID_ARGUMENT;
  switch (dtype) {
    case LLMOE_DTYPE_BF16:
    case LLMOE_DTYPE_FP16:
      if (out_dtype != dtype && out_dtype != LLMOE_DTYPE_FP32) return LLMOE_ERR_INVALID_ARGUMENT;
      break;
    case LLMOE_DTYPE_MX8:
      if (out_dtype == LLMOE_DTYPE_MX8 && !swiglu) return LLMOE_ERR_INVALID_ARGUMENT;
      break;
    default: return LLMOE_ERR_INVALID_ARGUMENT;
  }
  const uint64_t xr = row_bytes(in, dtype), yr = row_bytes(out, out_dtype);
  if (xr == 0 || yr == 0 || out > INT32_MAX / 2) return LLMOE_ERR_INVALID_ARGUMENT;
  if (x == nullptr || w == nullptr || y == nullptr || !aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) ||
      !aligned(counts, 8))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const uint64_t rows = (uint64_t)E * R * T, n = (uint64_t)out * (swiglu ? 2 : 1);
  const uint64_t limit = (uint64_t)INT64_MAX / 2;
  if (xr > limit / rows || yr > limit / rows || xr > limit / (n * E)) return LLMOE_ERR_INVALID_ARGUMENT;
  if (overlap(y, rows * yr, x, rows * xr) || overlap(y, rows * yr, w, n * E * xr)) return LLMOE_ERR_INVALID_ARGUMENT;
  *a = ProductArgs{};
  if (counts == nullptr) {
    const size_t total = llmoe_layout_bytes_dtype(T, bs->hidden, R, E, bs->dtype);
    uint64_t sig = 0;
    if (total == 0 || bs->base == nullptr || !aligned(bs->base, 16) || bs->rank_stride % 16 != 0 ||
        bs->rank_stride < total || bs->rank_stride > limit / R ||
        llmoe_layout_offsets_dtype(T, bs->hidden, R, E, bs->dtype, bs->set, nullptr, nullptr, &sig) != LLMOE_SUCCESS ||
        sig % 8 != 0)
      return LLMOE_ERR_INVALID_ARGUMENT;
    a->base = static_cast<const uint8_t*>(bs->base);
    a->rank_stride = bs->rank_stride;
    a->sig_off = sig;
  }
  a->x = static_cast<const uint8_t*>(x);
  a->w = static_cast<const uint8_t*>(w);
  a->y = static_cast<uint8_t*>(y);
  a->counts = counts;
  a->err = bs->err;
  a->T = T;
  a->R = R;
  a->E = E;
  a->L = E / R;
  a->in = in;
  a->out = out;
  a->n = (int)n;
  a->x_row = xr;
  a->y_row = yr;
  a->dtype = dtype;
  a->out_dtype = out_dtype;
  return LLMOE_SUCCESS;
}

}  // namespace

extern "C" int llmoe_expert_product(const void* x, const void* w, void* y, const int64_t* counts, int in_features,
                                    int out_features, int dtype, int out_dtype, uint32_t flags,
                                    const llmoe_buf_set_t* bs, llmoe_stream_t stream) {
  ProductArgs a;
  const int rc = product_args(x, w, y, counts, in_features, out_features, dtype, out_dtype, flags, bs, &a);
  if (rc != LLMOE_SUCCESS) return rc;
  const int64_t grid = (int64_t)a.E * ((a.out + kTile - 1) / kTile);
  if (grid > INT32_MAX) return LLMOE_ERR_INVALID_ARGUMENT;
  if ((flags & LLMOE_PRODUCT_SWIGLU) != 0) return launch_block(product_kernel<true>, (unsigned)grid, 256, 0, stream, a);
  return launch_block(product_kernel<false>, (unsigned)grid, 256, 0, stream, a);
}
