// block_weights.cu -- llmoe_pack_fp8b_weights (include/llmoe_block.h).
//
// A CTA takes one 128 x 128 block at a time: its values stay in registers (16-byte
// loads), the largest magnitude crosses the CTA, and the codes are stored from the
// registers, so that every byte is read and written once: HBM bounds it (32 matrices
// of 2048 x 7168 bf16: 218 us, 6.45 TB/s, 97% of the copy rate; 2000 x 1040 fp32 values
// 5.1 us, of which the call is most).
#include "block_common.cuh"

namespace {

struct WeightsArgs {
  const uint8_t* w;
  uint8_t* codes;
  float* scales;
  int64_t blocks;
  int rows, cols, down, across;  // blocks down and across a matrix
};

constexpr int kThreads = 256, kBlock = LLMOE_FP8B_BLOCK;

template <int DT>
__global__ void __launch_bounds__(kThreads) weights_kernel(WeightsArgs a) {
  constexpr int V = Quad<DT>::kValues, kBytes = 16 / V;
  constexpr int kLanes = kBlock / V, kRows = kThreads / kLanes, Q = kBlock / kRows;  // lanes a row, rows a pass, passes
  __shared__ uint32_t part[kThreads / 32];
  wait_prior_grid();
  release_next_grid();
  const int tid = threadIdx.x, r0 = tid / kLanes, c0 = tid % kLanes * V;
  for (int64_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    const int64_t line = b / a.across;  // of blocks, over all matrices
    const int col = (int)(b - line * a.across) * kBlock + c0, row = (int)(line % a.down) * kBlock + r0;
    const uint64_t at = ((uint64_t)(line / a.down) * a.rows + row) * a.cols + col, step = (uint64_t)kRows * a.cols;
    uint4 q[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i)
      q[i] = row + i * kRows < a.rows && col < a.cols ? *reinterpret_cast<const uint4*>(a.w + (at + i * step) * kBytes)
                                                      : make_uint4(0, 0, 0, 0);
    uint32_t most = 0;  // NaN above infinity above the rest
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      float v[V];
      unpack_quad<DT>(q[i], v);
#pragma unroll
      for (int k = 0; k < V; ++k) most = max(most, magnitude(v[k]));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    __syncthreads();  // the previous block's has been read
    if ((tid & 31) == 0) part[tid >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) most = max(most, part[i]);
    const float scale = block_scale(__uint_as_float(most)), inv = __frcp_rn(scale);
    if (tid == 0) a.scales[b] = scale;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      if (row + i * kRows >= a.rows || col >= a.cols) continue;
      float v[V];
      unpack_quad<DT>(q[i], v);
      uint32_t u[V / 4];
#pragma unroll
      for (int k = 0; k < V / 4; ++k)
        u[k] = pack_e4m3x2(v[4 * k] * inv, v[4 * k + 1] * inv) | pack_e4m3x2(v[4 * k + 2] * inv, v[4 * k + 3] * inv) << 16;
      uint8_t* to = a.codes + at + i * step;
      if constexpr (V == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(u[0], u[1]);
      else
        *reinterpret_cast<uint32_t*>(to) = u[0];
    }
  }
}

}  // namespace

extern "C" int llmoe_pack_fp8b_weights(const void* w, void* codes, float* scales, int64_t matrices, int rows, int cols,
                                       int dtype, llmoe_stream_t stream) {
  if ((dtype != LLMOE_DTYPE_BF16 && dtype != LLMOE_DTYPE_FP16 && dtype != LLMOE_DTYPE_FP32) || matrices < 0 ||
      rows < 1 || cols < 1 || cols % 16 != 0)
    return LLMOE_ERR_INVALID_ARGUMENT;
  const uint64_t n = (uint64_t)rows * cols, es = dtype == LLMOE_DTYPE_FP32 ? 4 : 2;
  if ((uint64_t)matrices > (uint64_t)INT64_MAX / 8 / n) return LLMOE_ERR_INVALID_ARGUMENT;
  if (matrices == 0) return LLMOE_SUCCESS;
  const int down = (int)(((int64_t)rows + kBlock - 1) / kBlock), across = (int)(((int64_t)cols + kBlock - 1) / kBlock);
  const int64_t blocks = matrices * down * across;
  if (w == nullptr || codes == nullptr || scales == nullptr || !aligned(w, 16) || !aligned(codes, 16) ||
      !aligned(scales, 4))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const uint64_t values = matrices * n, in = values * es, sb = (uint64_t)blocks * 4;
  if (overlap(codes, values, w, in) || overlap(scales, sb, w, in) || overlap(scales, sb, codes, values))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const WeightsArgs a{static_cast<const uint8_t*>(w), static_cast<uint8_t*>(codes), scales, blocks, rows, cols, down,
                      across};
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)num_sms() * 8);
  switch (dtype) {
    case LLMOE_DTYPE_FP16: return launch_block(weights_kernel<LLMOE_DTYPE_FP16>, grid, kThreads, 0, stream, a);
    case LLMOE_DTYPE_FP32: return launch_block(weights_kernel<LLMOE_DTYPE_FP32>, grid, kThreads, 0, stream, a);
    default: return launch_block(weights_kernel<LLMOE_DTYPE_BF16>, grid, kThreads, 0, stream, a);
  }
}
