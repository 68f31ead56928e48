"""An allocation that fails inside an entry point of the block pool or of cross
attention is an error code, not a C++ exception in the caller's C program."""
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
  void* m[10];
  for (auto& p : m)
    if (cudaMalloc(&p, 1 << 20) != cudaSuccess || cudaMemset(p, 0, 1 << 20) != cudaSuccess) return 2;
  cudaStream_t s[6];
  for (auto& x : s)
    if (cudaStreamCreate(&x) != cudaSuccess) return 2;
  int32_t* i[8];                               // zeros: rows of length 0, no request with a token
  for (int k = 0; k < 8; ++k) i[k] = static_cast<int32_t*>(m[k]);
  const size_t ws = cb_paged_cross_attention_workspace_size(1, 1, 1, 64, 4, 4, 64, 16);
  void* w = nullptr;
  if (cudaMalloc(&w, ws) != cudaSuccess) return 2;
  const size_t bytes[1] = {64};
  for (int pass = 0; pass < 2; ++pass) {
    fails = pass == 0;                         // each stream's first call makes the library's state of it
    int rc[5] = {cb_fork_blocks(i[0], nullptr, i[1], 4, 1, i[2], i[3], 4, 16, i[4], m[8], 1 << 20, s[0]),
                 cb_grow_blocks(i[0], i[1], 4, 1, i[2], i[3], 4, 16, i[4], static_cast<int64_t*>(m[5]), 3, m[8], 1 << 20, s[1]),
                 cb_compact_blocks(i[1], 4, 1, i[2], i[3], 4, 16, i[5], i[4], 2, i[6], m[8], 1 << 20, s[2]),
                 cb_copy_blocks_layers(i[0], 1, &m[9], bytes, 1, 1, 4, s[3]),
                 cb_paged_cross_attention(m[0], i[1], i[2], i[3], 4, 1, 1, 1, 64, m[5], m[6], 4, m[7], 0.1f, 4, 4, 64, 16, w, ws, s[4])};
    fails = false;
    for (int k = 0; k < 5; ++k) std::printf("%d ", rc[k]);
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
