// block_common.cuh -- what the translation units of llmoe_block.h share: host
// checks and launch, 16-byte rows as fp32 values, MX8 and FP8B encoding.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "llmoe_block.h"

namespace {

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlap(const void* a, uint64_t an, const void* b, uint64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// Streaming multiprocessors of the current device (atomic per device: host
// threads may call concurrently, and two that miss together store the same).
inline int num_sms() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
  if (dev < kMaxDevices) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Launches with programmatic stream serialization, as the data-path kernels
// do: every kernel waits for the previous grid before its first global access.
template <typename... KArgs, typename... Args>
int launch_block(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, llmoe_stream_t stream,
                 Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) != cudaSuccess) {
    cudaGetLastError();  // clear the launch error so it does not leak into later calls
    return LLMOE_ERR_CUDA;
  }
  return LLMOE_SUCCESS;
}

// Bytes of a row of n values, 0 where there is no such row (llmoe_row_bytes).
inline uint64_t row_bytes(int64_t n, int dtype) {
  if (n < 1) return 0;
  switch (dtype) {
    case LLMOE_DTYPE_BF16:
    case LLMOE_DTYPE_FP16: return n % 8 == 0 ? (uint64_t)n * 2 : 0;
    case LLMOE_DTYPE_FP32: return n % 4 == 0 ? (uint64_t)n * 4 : 0;
    case LLMOE_DTYPE_MX8: return n % 32 == 0 ? (uint64_t)n + (uint64_t)(n / 32 + 15) / 16 * 16 : 0;
    case LLMOE_DTYPE_FP8B:
      return n % 16 == 0 ? (uint64_t)n + ((uint64_t)(n + LLMOE_FP8B_BLOCK - 1) / LLMOE_FP8B_BLOCK * 4 + 15) / 16 * 16 : 0;
    default: return 0;
  }
}

// ---------------------------------------------------------------------------
// device side
// ---------------------------------------------------------------------------
// A kernel here lets the next one on the stream start (release_next_grid) only
// after its own wait: whatever starts behind it then finds everything before
// it complete, among it a router's topk_idx and topk_w for a combine that
// reads them before its wait (LLMOE_FLAG_INPUTS_READY).  Releasing before the
// wait measured the same on every call (one-token norm 5.8 us, router 6.3,
// smallest product 7.3), large norm 64.4 against 64.2 us.  And no load is
// through a __restrict__ pointer or __ldg: the compiler would be free to move
// it before the wait, and a read-only load must not meet memory that is still
// written while the kernel starts.  Plain loads measured the same.
__device__ __forceinline__ void wait_prior_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void release_next_grid() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void report(int32_t* err, int32_t code) {
  if (err != nullptr) atomicCAS(err, 0, code);
}

// A 16-byte quad of values: 8 of bf16 / fp16, 4 of fp32.
template <int DT>
struct Quad {
  static constexpr int kValues = DT == LLMOE_DTYPE_FP32 ? 4 : 8;
};

template <int DT>
__device__ __forceinline__ void unpack_quad(const uint4& q, float (&v)[Quad<DT>::kValues]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == LLMOE_DTYPE_FP32) {
      v[i] = __uint_as_float(u[i]);
    } else if constexpr (DT == LLMOE_DTYPE_FP16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    } else {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack_quad(const float (&v)[Quad<DT>::kValues]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == LLMOE_DTYPE_FP32) {
      u[i] = __float_as_uint(v[i]);
    } else if constexpr (DT == LLMOE_DTYPE_FP16) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// |v| as an integer that orders like the magnitude, a NaN above infinity: the
// maximum of these over a group finds its largest value or its NaN.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The e8m0 scale code of a group from its largest magnitude: the smallest s
// with amax <= 448 * 2^(s - 127).  448 = 1.75 * 2^8, so with amax = m * 2^q
// s - 127 = q - 8, one more when m > 1.75 (the addition below carries into the
// exponent exactly then).  At least 1 (scale 2^-126, so that its inverse is a
// normal float); 255, the NaN scale, when the group holds an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255;
  const int s = (int)((amax + 0x1fffffu) >> 23) - 8;
  return s < 1 ? 1u : (uint32_t)s;
}
// 1 / scale, exactly: 2^(127 - code); code is at most 247 for a finite group.
__device__ __forceinline__ float scale_inverse(uint32_t code) {
  return code == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - code) << 23);
}
// The FP8B scale of a block whose largest magnitude is amax (NaN where the block
// holds one): NaN where it is not finite; the codes are of v * (1 / scale).  The
// least scale is a normal float with a finite inverse.
__device__ __forceinline__ float block_scale(float amax) {
  if (!(amax < INFINITY)) return __uint_as_float(0x7fffffffu);
  return fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-126f);
}
// Two quotients as e4m3 (nearest even; none rounds to more than 448), a in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace
