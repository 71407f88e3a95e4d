// block_rows.cu -- llmoe_add_rmsnorm, llmoe_pack_mx8 and llmoe_row_bytes
// (include/llmoe_block.h).
//
// One CTA holds one row at a time in registers: 16-byte loads of x and
// residual, h = T(x + residual), the sum of squares over the CTA in fp32, then
// v = h * r * weight from the registers and 16-byte (MX8: 8-byte) stores.
// Every byte is read and written once, so HBM bandwidth bounds it (a few
// operations per byte).
#include "block_common.cuh"

namespace {

struct RowsArgs {
  const uint4* x;
  const uint4* residual;  // or null
  const uint4* weight;    // null: no norm (llmoe_pack_mx8)
  uint4* residual_out;    // or null
  uint8_t* out;
  int64_t rows;
  float eps, inv_n;
  int hidden, nq;       // values and 16-byte quads per row of T
  uint64_t out_stride;  // bytes of an output row
};

__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  __syncthreads();  // the previous row's sums have been read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// DT: T of x, residual, weight; MX: MX8 output rows; Q: quads per thread.
template <int DT, bool MX, int Q>
__global__ void __launch_bounds__(1024) rows_kernel(RowsArgs a) {
  constexpr int V = Quad<DT>::kValues;
  constexpr int kLanes = 32 / V;  // adjacent lanes that hold one group of 32
  __shared__ float part[32];
  release_next_grid();
  wait_prior_grid();
  const int tid = threadIdx.x, nthr = blockDim.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float h[Q][V];
    const uint4* x = a.x + row * a.nq;
    uint4 in[Q], res[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int j = tid + i * nthr;
      in[i] = j < a.nq ? x[j] : make_uint4(0, 0, 0, 0);
      if (a.residual != nullptr) res[i] = j < a.nq ? a.residual[row * a.nq + j] : make_uint4(0, 0, 0, 0);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int j = tid + i * nthr;
      unpack_quad<DT>(in[i], h[i]);
      if (a.residual != nullptr) {
        float r[V];
        unpack_quad<DT>(res[i], r);
#pragma unroll
        for (int k = 0; k < V; ++k) h[i][k] += r[k];
        const uint4 q = pack_quad<DT>(h[i]);  // the norm is of the rounded sum
        unpack_quad<DT>(q, h[i]);
        in[i] = q;
      }
      if (a.residual_out != nullptr && j < a.nq) a.residual_out[row * a.nq + j] = in[i];
#pragma unroll
      for (int k = 0; k < V; ++k) sum += h[i][k] * h[i][k];
    }
    if (a.weight != nullptr) {
      const float r = 1.0f / sqrtf(block_sum(sum, part) * a.inv_n + a.eps);
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int j = tid + i * nthr;
        float w[V];
        unpack_quad<DT>(j < a.nq ? __ldg(a.weight + j) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
        for (int k = 0; k < V; ++k) h[i][k] = h[i][k] * r * w[k];
      }
    }
    uint8_t* out = a.out + row * a.out_stride;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int j = tid + i * nthr;
      if constexpr (MX) {
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) amax = max(amax, magnitude(h[i][k]));
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        const uint32_t code = scale_code(amax);
        const float inv = scale_inverse(code);
        if (j < a.nq) {
          uint32_t b[V / 4];
#pragma unroll
          for (int k = 0; k < V / 4; ++k)
            b[k] = pack_e4m3x2(h[i][4 * k] * inv, h[i][4 * k + 1] * inv) |
                   pack_e4m3x2(h[i][4 * k + 2] * inv, h[i][4 * k + 3] * inv) << 16;
          if constexpr (V == 8)
            *reinterpret_cast<uint2*>(out + (size_t)j * 8) = make_uint2(b[0], b[1]);
          else
            *reinterpret_cast<uint32_t*>(out + (size_t)j * 4) = b[0];
          if (j % kLanes == 0) out[a.hidden + j / kLanes] = (uint8_t)code;
        }
      } else {
        if (j < a.nq) reinterpret_cast<uint4*>(out)[j] = pack_quad<DT>(h[i]);
      }
    }
    if constexpr (MX) {  // zeros up to the row's 16-byte end
      const int used = a.hidden + a.hidden / 32;
      if (tid < (int)a.out_stride - used) out[used + tid] = 0;
    }
  }
}

template <int DT, bool MX>
int launch_rows(const RowsArgs& a, llmoe_stream_t stream) {
  const int64_t sms = num_sms();
  const unsigned grid = (unsigned)std::min<int64_t>(a.rows, sms * 8);
  // one to eight quads per thread, CTAs of 128 threads and up
  int threads = 128;
  while (threads < 1024 && threads * 4 < a.nq) threads *= 2;
  const int q = (a.nq + threads - 1) / threads;
  if (q <= 1) return launch_block(rows_kernel<DT, MX, 1>, grid, threads, 0, stream, a);
  if (q <= 2) return launch_block(rows_kernel<DT, MX, 2>, grid, threads, 0, stream, a);
  if (q <= 4) return launch_block(rows_kernel<DT, MX, 4>, grid, threads, 0, stream, a);
  return launch_block(rows_kernel<DT, MX, 8>, grid, threads, 0, stream, a);
}

template <bool MX>
int launch_rows_dtype(const RowsArgs& a, int dtype, llmoe_stream_t stream) {
  switch (dtype) {
    case LLMOE_DTYPE_FP16: return launch_rows<LLMOE_DTYPE_FP16, MX>(a, stream);
    case LLMOE_DTYPE_FP32: return launch_rows<LLMOE_DTYPE_FP32, MX>(a, stream);
    default: return launch_rows<LLMOE_DTYPE_BF16, MX>(a, stream);
  }
}

// Fills the geometry of a call on `rows` rows of `hidden` values; false where
// the arguments are not valid.
bool rows_geometry(const void* x, const void* out, int64_t rows, int hidden, int dtype, int out_dtype, RowsArgs* a) {
  if (dtype != LLMOE_DTYPE_BF16 && dtype != LLMOE_DTYPE_FP16 && dtype != LLMOE_DTYPE_FP32) return false;
  const uint64_t rb = row_bytes(hidden, dtype), ob = row_bytes(hidden, out_dtype);
  if (rb == 0 || ob == 0 || hidden > LLMOE_MAX_ROW_VALUES || rows < 0 || rows > INT64_MAX / 2 / (int64_t)std::max(rb, ob))
    return false;
  if (rows > 0 && (x == nullptr || out == nullptr || !aligned(x, 16) || !aligned(out, 16))) return false;
  *a = RowsArgs{};
  a->x = static_cast<const uint4*>(x);
  a->out = static_cast<uint8_t*>(const_cast<void*>(out));
  a->rows = rows;
  a->hidden = hidden;
  a->nq = (int)(rb / 16);
  a->out_stride = ob;
  return true;
}

}  // namespace

extern "C" {

size_t llmoe_row_bytes(int n, int dtype) { return (size_t)row_bytes(n, dtype); }

int llmoe_pack_mx8(const void* x, void* out, int64_t rows, int hidden, int dtype, llmoe_stream_t stream) {
  RowsArgs a;
  if (!rows_geometry(x, out, rows, hidden, dtype, LLMOE_DTYPE_MX8, &a)) return LLMOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return LLMOE_SUCCESS;
  if (overlap(x, (uint64_t)rows * a.nq * 16, out, (uint64_t)rows * a.out_stride)) return LLMOE_ERR_INVALID_ARGUMENT;
  return launch_rows_dtype<true>(a, dtype, stream);
}

int llmoe_add_rmsnorm(const void* x, const void* residual, const void* weight, float eps, void* residual_out,
                      void* out, int64_t rows, int hidden, int dtype, int out_dtype, llmoe_stream_t stream) {
  RowsArgs a;
  if ((out_dtype != dtype && out_dtype != LLMOE_DTYPE_MX8) || !(eps >= 0.0f) ||
      !rows_geometry(x, out, rows, hidden, dtype, out_dtype, &a))
    return LLMOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return LLMOE_SUCCESS;
  if (weight == nullptr || !aligned(weight, 16) || !aligned(residual, 16) || !aligned(residual_out, 16))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const uint64_t n = (uint64_t)a.nq * 16, in_bytes = (uint64_t)rows * n, out_bytes = (uint64_t)rows * a.out_stride;
  // rows are read before they are written and never again, so a row may
  // replace itself; any other overlap is refused
  const bool out_is_x = out == x && out_dtype == dtype;
  if ((!out_is_x && overlap(out, out_bytes, x, in_bytes)) || overlap(out, out_bytes, weight, n) ||
      (residual != nullptr && overlap(out, out_bytes, residual, in_bytes)))
    return LLMOE_ERR_INVALID_ARGUMENT;
  if (residual_out != nullptr &&
      (overlap(residual_out, in_bytes, out, out_bytes) || overlap(residual_out, in_bytes, weight, n) ||
       (residual_out != x && overlap(residual_out, in_bytes, x, in_bytes)) ||
       (residual != nullptr && residual_out != residual && overlap(residual_out, in_bytes, residual, in_bytes))))
    return LLMOE_ERR_INVALID_ARGUMENT;
  a.residual = static_cast<const uint4*>(residual);
  a.weight = static_cast<const uint4*>(weight);
  a.residual_out = static_cast<uint4*>(residual_out);
  a.eps = eps;
  a.inv_n = 1.0f / (float)hidden;
  return out_dtype == LLMOE_DTYPE_MX8 ? launch_rows_dtype<true>(a, dtype, stream)
                                      : launch_rows_dtype<false>(a, dtype, stream);
}

}  // extern "C"
