// block_rows.cu -- llmoe_add_rmsnorm, llmoe_pack_mx8, llmoe_pack_fp8b and llmoe_row_bytes
// (include/llmoe_block.h).
//
// One CTA holds one row at a time in registers: 16-byte loads of x and
// residual, h = T(x + residual), the sum of squares over the CTA in fp32, then
// v = h * r * weight from the registers and 16-byte (MX8: 8-byte) stores.
// Every byte is read and written once, so HBM bandwidth bounds a large call
// (8192 rows of 7168 bf16 with a residual to MX8: 63.2 us, 6.5 TB/s, 98% of the
// copy rate; to FP8B 63.7, 97%; to bf16 75.5 us, 93%), launch and load latency a small one (one row
// 2.2 us, 1024 rows 11.0).  A few large CTAs per SM stay for all rows and load the
// next row into the registers that the sum has just freed: 1024 rows 11.0 us against 12.6 with
// the next row prefetched into L2, and 12.7 with a CTA per row.  Two quads a
// thread rather than four: 152 rows 3.1 us against 4.3.  Rows of more than 2048
// quads take four or, fp32, eight a thread, which spill under 64 registers: 32768
// bf16 values 92% of the copy rate, 16384 fp32 95%, 32768 fp32 57% (to MX8 76, 89
// and 29%).  Sums are packed additions of T and the fp32 arithmetic is on pairs.
#include "block_common.cuh"

namespace {

struct RowsArgs {
  const uint4* x;
  const uint4* residual;  // or null
  const uint4* weight;    // null for llmoe_pack_mx8 and llmoe_pack_fp8b
  uint4* residual_out;    // or null
  uint8_t* out;
  int64_t rows;
  float eps, inv_n;
  int hidden, nq;       // values and 16-byte quads per row of T
  uint64_t out_stride;  // bytes of an output row
};

// Pairs of fp32 values in one register pair: one instruction for both.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ float2 unpair(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// The larger magnitude; NaN where either is.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}

template <int DT>
__device__ __forceinline__ void quad_pairs(const uint4& q, Pair (&p)[Quad<DT>::kValues / 2]) {
  float v[Quad<DT>::kValues];
  unpack_quad<DT>(q, v);
#pragma unroll
  for (int i = 0; i < Quad<DT>::kValues / 2; ++i) p[i] = pair(v[2 * i], v[2 * i + 1]);
}

// T(a + b).  The packed additions round the exact sum to T once; the fp32 sum
// rounded to T is the same: with 8 (11) significant bits each, either the fp32
// sum is exact or the smaller operand is too small to reach a rounding boundary.
template <int DT>
__device__ __forceinline__ uint4 add_quad(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == LLMOE_DTYPE_FP32) {
      u[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(y[i]));
    } else if constexpr (DT == LLMOE_DTYPE_FP16) {
      const __half2 h = __hadd2_rn(*reinterpret_cast<const __half2*>(&x[i]), *reinterpret_cast<const __half2*>(&y[i]));
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&x[i]),
                                          *reinterpret_cast<const __nv_bfloat162*>(&y[i]));
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

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

// DT: T of x, residual, weight; OUT: DT, or MX8 or FP8B output rows; Q: quads
// per thread; kNorm: false for llmoe_pack_mx8 and llmoe_pack_fp8b.
template <int DT, int OUT, int Q, bool kNorm>
__global__ void __launch_bounds__(1024) rows_kernel(RowsArgs a) {
  constexpr int V = Quad<DT>::kValues, P = V / 2;
  constexpr bool MX = OUT == LLMOE_DTYPE_MX8, k8Bit = MX || OUT == LLMOE_DTYPE_FP8B;
  constexpr int kLanes = (MX ? 32 : LLMOE_FP8B_BLOCK) / V;  // adjacent lanes that hold one scale's values
  __shared__ float part[32];
  wait_prior_grid();
  release_next_grid();
  const int tid = threadIdx.x, nthr = blockDim.x;
  uint4 x[Q], res[Q];  // the next row to be normed
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int j = tid + i * nthr;
      x[i] = j < a.nq ? a.x[row * a.nq + j] : make_uint4(0, 0, 0, 0);
      if (kNorm && a.residual != nullptr) res[i] = j < a.nq ? a.residual[row * a.nq + j] : make_uint4(0, 0, 0, 0);
    }
  };
  int64_t row = blockIdx.x;
  if (row < a.rows) load(row);
  for (; row < a.rows; row += gridDim.x) {
    uint4 h[Q];
    Pair sum = 0;  // of squares
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      h[i] = x[i];
      if constexpr (kNorm) {
        const int j = tid + i * nthr;
        if (a.residual != nullptr) h[i] = add_quad<DT>(h[i], res[i]);  // the norm is of the rounded sum
        if (a.residual_out != nullptr && j < a.nq) a.residual_out[row * a.nq + j] = h[i];
        Pair v[P];
        quad_pairs<DT>(h[i], v);
#pragma unroll
        for (int k = 0; k < P; ++k) sum = fma2(v[k], v[k], sum);
      }
    }
    // its registers are free: the next row is on its way while this one's sum
    // crosses the CTA and its output is written
    if (row + gridDim.x < a.rows) load(row + gridDim.x);
    Pair r2 = 0;
    if constexpr (kNorm) {
      const float2 s = unpair(sum);
      const float r = 1.0f / sqrtf(block_sum(s.x + s.y, part) * a.inv_n + a.eps);
      r2 = pair(r, r);
    }
    uint8_t* out = a.out + row * a.out_stride;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int j = tid + i * nthr;
      if (Q > 1 && (j & ~31) >= a.nq) break;  // the warp's quads are past the row
      Pair v[P];
      quad_pairs<DT>(h[i], v);
      if constexpr (kNorm) {
        Pair w[P];
        quad_pairs<DT>(j < a.nq ? a.weight[j] : make_uint4(0, 0, 0, 0), w);
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = mul2(mul2(v[k], r2), w[k]);
      }
      if constexpr (k8Bit) {
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const float2 f = unpair(v[k]);
          most = max_magnitude(max_magnitude(most, f.x), f.y);
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) most = max_magnitude(most, __shfl_xor_sync(0xffffffffu, most, d));
        // the scale, as an e8m0 code or a float, and its inverse
        const uint32_t scale = MX ? scale_code(__float_as_uint(most)) : __float_as_uint(block_scale(most));
        const float inv = MX ? scale_inverse(scale) : __frcp_rn(__uint_as_float(scale));
        const Pair inv2 = pair(inv, inv);
        if (j < a.nq) {
          uint32_t b[P];
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const float2 f = unpair(mul2(v[k], inv2));
            b[k] = pack_e4m3x2(f.x, f.y);
          }
          if constexpr (V == 8)
            *reinterpret_cast<uint2*>(out + (size_t)j * 8) =
                make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
          else
            *reinterpret_cast<uint32_t*>(out + (size_t)j * 4) = __byte_perm(b[0], b[1], 0x5410);
          if (j % kLanes == 0) {
            if constexpr (MX)
              out[a.hidden + j / kLanes] = (uint8_t)scale;
            else
              reinterpret_cast<uint32_t*>(out + a.hidden)[j / kLanes] = scale;
          }
        }
      } else if (j < a.nq) {
        float f[V];
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const float2 g = unpair(v[k]);
          f[2 * k] = g.x;
          f[2 * k + 1] = g.y;
        }
        reinterpret_cast<uint4*>(out)[j] = pack_quad<DT>(f);
      }
    }
    if constexpr (k8Bit) {  // zeros up to the row's 16-byte end
      const int used = a.hidden + (MX ? a.hidden / 32 : (a.hidden + LLMOE_FP8B_BLOCK - 1) / LLMOE_FP8B_BLOCK * 4);
      if (tid < (int)a.out_stride - used) out[used + tid] = 0;
    }
  }
}

template <int DT, int OUT, bool kNorm>
int launch_rows(const RowsArgs& a, llmoe_stream_t stream) {
  // two quads per thread where a CTA has threads enough; as many CTAs as the
  // registers (64 a thread) hold
  const int threads = std::min(1024, std::max(128, ((a.nq + 1) / 2 + 31) / 32 * 32));
  const unsigned grid = (unsigned)std::min<int64_t>(a.rows, (int64_t)num_sms() * (1024 / threads));
  const int q = (a.nq + threads - 1) / threads;
  if (q <= 1) return launch_block(rows_kernel<DT, OUT, 1, kNorm>, grid, threads, 0, stream, a);
  if (q <= 2) return launch_block(rows_kernel<DT, OUT, 2, kNorm>, grid, threads, 0, stream, a);
  if constexpr (DT == LLMOE_DTYPE_FP32)  // 16-bit rows have at most four quads for each of 1024 threads
    if (q > 4) return launch_block(rows_kernel<DT, OUT, 8, kNorm>, grid, threads, 0, stream, a);
  static_assert(LLMOE_MAX_ROW_VALUES <= 4 * 1024 * 8, "16-bit rows past four quads a thread");
  return launch_block(rows_kernel<DT, OUT, 4, kNorm>, grid, threads, 0, stream, a);
}

// OUT: MX8 or FP8B rows, or (BF16) rows of the input's type.
template <int OUT, bool kNorm>
int launch_rows_dtype(const RowsArgs& a, int dtype, llmoe_stream_t stream) {
  constexpr bool k8Bit = OUT == LLMOE_DTYPE_MX8 || OUT == LLMOE_DTYPE_FP8B;
  switch (dtype) {
    case LLMOE_DTYPE_FP16: return launch_rows<LLMOE_DTYPE_FP16, k8Bit ? OUT : LLMOE_DTYPE_FP16, kNorm>(a, stream);
    case LLMOE_DTYPE_FP32: return launch_rows<LLMOE_DTYPE_FP32, k8Bit ? OUT : LLMOE_DTYPE_FP32, kNorm>(a, stream);
    default: return launch_rows<LLMOE_DTYPE_BF16, k8Bit ? OUT : LLMOE_DTYPE_BF16, kNorm>(a, stream);
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

template <int OUT>
int pack_rows(const void* x, void* out, int64_t rows, int hidden, int dtype, llmoe_stream_t stream) {
  RowsArgs a;
  if (!rows_geometry(x, out, rows, hidden, dtype, OUT, &a)) return LLMOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return LLMOE_SUCCESS;
  if (overlap(x, (uint64_t)rows * a.nq * 16, out, (uint64_t)rows * a.out_stride)) return LLMOE_ERR_INVALID_ARGUMENT;
  return launch_rows_dtype<OUT, false>(a, dtype, stream);
}

}  // namespace

extern "C" {

size_t llmoe_row_bytes(int n, int dtype) { return (size_t)row_bytes(n, dtype); }

int llmoe_pack_mx8(const void* x, void* out, int64_t rows, int hidden, int dtype, llmoe_stream_t stream) {
  return pack_rows<LLMOE_DTYPE_MX8>(x, out, rows, hidden, dtype, stream);
}

int llmoe_pack_fp8b(const void* x, void* out, int64_t rows, int hidden, int dtype, llmoe_stream_t stream) {
  return pack_rows<LLMOE_DTYPE_FP8B>(x, out, rows, hidden, dtype, stream);
}

int llmoe_add_rmsnorm(const void* x, const void* residual, const void* weight, float eps, void* residual_out,
                      void* out, int64_t rows, int hidden, int dtype, int out_dtype, llmoe_stream_t stream) {
  RowsArgs a;
  if ((out_dtype != dtype && out_dtype != LLMOE_DTYPE_MX8 && out_dtype != LLMOE_DTYPE_FP8B) || !(eps >= 0.0f) ||
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
  switch (out_dtype) {
    case LLMOE_DTYPE_MX8: return launch_rows_dtype<LLMOE_DTYPE_MX8, true>(a, dtype, stream);
    case LLMOE_DTYPE_FP8B: return launch_rows_dtype<LLMOE_DTYPE_FP8B, true>(a, dtype, stream);
    default: return launch_rows_dtype<LLMOE_DTYPE_BF16, true>(a, dtype, stream);
  }
}

}  // extern "C"
