"""GPU test of the router's reciprocal (one_over, csrc/block_router.cuh): equal to
CUDA's __frcp_rn on its whole range, all floats of [1, 2^126].  The choice of
experts depends on it: keys of tokens that take it and of those that take the
general reciprocal have to order alike."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "block_router.cuh"

// Where one_over(d) is not __frcp_rn(d), d's bits from first to last: how many, and the least.
__global__ void compare_kernel(uint32_t first, uint32_t last, unsigned long long* bad, uint32_t* least) {
  const uint64_t step = (uint64_t)gridDim.x * blockDim.x;
  for (uint64_t i = first + (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i <= last; i += step) {
    const float d = __uint_as_float((uint32_t)i);
    if (__float_as_uint(one_over(d)) != __float_as_uint(__frcp_rn(d))) {
      atomicAdd(bad, 1ull);
      atomicMin(least, (uint32_t)i);
    }
  }
}

extern "C" __attribute__((visibility("default"))) int compare(uint32_t first, uint32_t last, unsigned long long* bad,
                                                              uint32_t* least) {
  compare_kernel<<<1216, 256>>>(first, last, bad, least);
  return (int)cudaGetLastError();
}
"""


def bits(v):
    return int(np.float32(v).view(np.uint32))


def test_reciprocal_is_the_rounded_one(tmp_path):
    from combine_routing_count_prefix_gb300 import build

    src, so = tmp_path / "compare.cu", tmp_path / "compare.so"
    src.write_text(SOURCE)
    subprocess.run([build.nvcc(), *build.NVCC_FLAGS, "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), "-o",
                    str(so), str(src)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.compare.argtypes = [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p]
    bad = torch.zeros(1, dtype=torch.int64, device="cuda")
    least = torch.full((1,), -1, dtype=torch.int32, device="cuda")  # the largest unsigned
    assert 1 + np.exp(87.0) < 2.0 ** 126  # what a logit of -87 asks for
    torch.cuda.synchronize()
    assert lib.compare(bits(1.0), bits(2.0 ** 126), bad.data_ptr(), least.data_ptr()) == 0
    torch.cuda.synchronize()
    assert int(bad) == 0, (int(bad), hex(int(least) & 0xFFFFFFFF))
