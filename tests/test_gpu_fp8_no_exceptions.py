"""An allocation that fails inside an entry point of the 8-bit cache is an error
code, not a C++ exception in the caller's C program."""
import os
import shutil
import subprocess

import pytest
import torch

from gpu_util import L

pytestmark = pytest.mark.gpu

SRC = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include <cuda_runtime.h>
#include "cbattn.h"
static bool fails = false;
void* operator new(size_t n) {
  if (fails) throw std::bad_alloc();
  return std::malloc(n ? n : 1);
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }
int main() {
  void* m[8];
  for (auto& p : m)
    if (cudaMalloc(&p, 1 << 20) != cudaSuccess || cudaMemset(p, 0, 1 << 20) != cudaSuccess) return 2;
  cudaStream_t s[6];
  for (auto& x : s)
    if (cudaStreamCreate(&x) != cudaSuccess) return 2;
  auto slots = static_cast<int64_t*>(m[6]);
  auto ints = static_cast<int32_t*>(m[6]);   // zeros: no request has a token
  const size_t ws = cb_paged_attention_fp8_workspace_size(1, 1, 1, 64, 4, 4, 64, 16);
  void* w = nullptr;
  if (cudaMalloc(&w, ws) != cudaSuccess) return 2;
  for (int pass = 0; pass < 2; ++pass) {
    fails = pass == 0;                         // each stream's first call makes the library's state of it
    int rc[5] = {
        cb_kv_append_fp8(m[0], m[1], slots, 1, m[2], m[3], m[4], m[5], 4, 4, 64, 16, s[0]),
        cb_kv_gather_fp8(slots, 1, m[2], m[3], m[4], m[5], 4, m[0], m[1], 4, 64, 16, s[1]),
        cb_copy_blocks_fp8(ints, 1, m[2], m[3], m[4], m[5], 4, 4, 64, 16, s[2]),
        cb_paged_attention_fp8(m[0], ints, ints, ints, 4, 1, 1, 1, 64, m[2], m[3], m[4], m[5], 4, m[7], 0.1f, 4, 4, 64, 16, 0, w, ws, s[3]),
        cb_kv_append_paged_attention_fp8(m[0], m[1], slots, m[0], ints, ints, ints, 4, 1, 1, 1, 64, m[2], m[3], m[4], m[5], 4, m[7], 0.1f,
                                         4, 4, 64, 16, 0, w, ws, s[4])};
    fails = false;
    for (int i = 0; i < 5; ++i) std::printf("%d ", rc[i]);
  }
  std::printf("%d\n", (int)cudaDeviceSynchronize());
  return 0;
}
"""


def test_a_failing_allocation_is_an_error_code(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = L()
    lib.lib()
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    here, root = os.path.dirname(lib.LIB_PATH), os.path.dirname(os.path.dirname(lib.LIB_PATH))
    (tmp_path / "t.cpp").write_text(SRC)
    subprocess.run([nvcc, "-std=c++17", "-I", os.path.join(root, "include"), str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t"),
                    lib.LIB_PATH, "-Xlinker", "-rpath", "-Xlinker", here], check=True)
    out = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == ["-2"] * 5 + ["0"] * 6
