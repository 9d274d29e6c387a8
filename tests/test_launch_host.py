"""The launch helpers of the C entry points on the host: no exception leaves them."""
import subprocess

from dynamic_layer_wise_b200 import build

# Stands in for the runtime's two calls, so no device is needed or touched.
PROGRAM = r"""
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdio>
static int g_calls = 0;
static cudaError_t fake_device(int *d) { *d = 0; return cudaSuccess; }
static cudaError_t fake_attribute(const void *, cudaFuncAttribute, int) { ++g_calls; return cudaSuccess; }
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_attribute
#include "dynamic_layer_wise_b200/csrc/common.cuh"
extern bool g_full;
int main() {
  static int kern;
  g_full = true;
  try {
    dcu::prefer_max_smem(&kern);
  } catch (...) {
    std::puts("threw");
    return 1;
  }
  g_full = false;
  dcu::prefer_max_smem(&kern);  // not recorded before: asked for again, and now recorded
  dcu::prefer_max_smem(&kern);
  std::printf("calls %d\n", g_calls);
  return g_calls == 2 ? 0 : 1;
}
"""

# An allocator that has no memory while g_full is set.
ALLOCATOR = r"""
#include <cstdlib>
#include <new>
bool g_full = false;
void *operator new(std::size_t n) {
  void *p = g_full ? nullptr : std::malloc(n);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
"""


def test_no_exception_leaves_a_launch_without_memory(tmp_path):
    src, alloc, exe = tmp_path / "launch.cu", tmp_path / "alloc.cpp", tmp_path / "launch"
    src.write_text(PROGRAM)
    alloc.write_text(ALLOCATOR)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", build.ROOT, "-o", str(exe), str(src), str(alloc)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout)
