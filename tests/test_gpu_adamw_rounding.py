"""The AdamW step's own root and reciprocal, bit by bit against CUDA's rounded ones, over every
float that they are given: roots of all floats from 0 up, inverses of 2^-100 to 2^14 (a block's
largest magnitude on the fast path of encode8)."""
import os
import subprocess

import pytest

from forward_moe_route_b200 import build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <cstdio>
#include "adamw.cuh"
using namespace moe::adamw;

// the number of floats with bits first .. last whose root, or inverse, differs; eight at a time
// are neighbours, or (apart > 0) come from places so far apart that large and tiny ones meet
__global__ void k_roots(uint32_t first, uint32_t last, uint32_t apart, unsigned long long* off) {
  const uint32_t n = last - first + 1, step = 8 * gridDim.x * blockDim.x;
  for (uint32_t i = 8 * (blockIdx.x * blockDim.x + threadIdx.x); i < n; i += step) {
    float v[8], root[8];
    float most = 0.f;
    for (int j = 0; j < 8; ++j) {
      v[j] = __uint_as_float(first + (apart ? (uint32_t)(((unsigned long long)i + j * apart) % n)
                                            : min(i + j, n - 1)));
      most = fmaxf(most, __fsqrt_rn(v[j]));
    }
    const float got = roots8(v, root);
    for (int j = 0; j < 8; ++j)
      if (__float_as_uint(root[j]) != __float_as_uint(__fsqrt_rn(v[j]))) atomicAdd(off, 1);
    if (got != most) atomicAdd(off, 1);
  }
}
__global__ void k_inverses(uint32_t first, uint32_t last, unsigned long long* off) {
  const uint32_t n = last - first + 1;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    const float x = __uint_as_float(first + i);
    if (__float_as_uint(inverse_step(x)) != __float_as_uint(__frcp_rn(x))) atomicAdd(off, 1);
  }
}

int main() {
  unsigned long long *off, h[3];
  if (cudaMalloc(&off, 24) != cudaSuccess || cudaMemset(off, 0, 24) != cudaSuccess) return 1;
  k_roots<<<592, 256>>>(0u, 0x7f7fffffu, 0u, off);
  k_roots<<<592, 256>>>(0u, 0x7f7fffffu, 0x0ffffff1u, off + 1);
  k_inverses<<<592, 256>>>(0x0d800000u, 0x46800000u, off + 2);
  if (cudaMemcpy(h, off, 24, cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
  printf("%llu %llu %llu\n", h[0], h[1], h[2]);
  return 0;
}
"""


def test_roots_and_inverses_are_rounded(tmp_path):
    source, exe = tmp_path / "rounding.cu", tmp_path / "rounding"
    source.write_text(SOURCE)
    flags = [f for f in build.FLAGS if f not in ("-Xcompiler", "-fPIC", "-shared")]
    subprocess.run([build.NVCC, *flags, "-I", build.SRC, "-o", os.fspath(exe), os.fspath(source)],
                   check=True)
    out = subprocess.run([os.fspath(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.split() == ["0", "0", "0"]
