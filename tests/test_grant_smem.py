"""Two host threads whose first calls of one kernel need different amounts of
shared memory: whatever their order, the kernel's limit ends up enough for both.
The CUDA runtime is a fake (the process has no device); the thread with the
smaller need sets its limit last."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = "/usr/local/cuda/include"

SOURCE = r"""
#include <atomic>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>

#include <cuda_runtime.h>
// the typed forms, which the headers give to nvcc alone
template <class T> cudaError_t cudaFuncSetAttribute(T* f, cudaFuncAttribute a, int v) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(f), a, v);
}
template <class T> cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, T* f) {
  return cudaFuncGetAttributes(a, reinterpret_cast<const void*>(f));
}

#include "internal.h"

constexpr int kOptin = 232448, kStatic = 64, kSmall = 60000, kLarge = 150000;
std::mutex mu;
std::condition_variable cv;
bool small_inside = false, large_done = false;
int limit = 49152, sets = 0;
thread_local bool is_small = false;

extern "C" cudaError_t cudaFuncSetAttribute(const void*, enum cudaFuncAttribute attr, int value) {
  if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
  if (value + kStatic > kOptin) return cudaErrorInvalidValue;
  std::unique_lock<std::mutex> lock(mu);
  if (is_small) {
    small_inside = true;
    cv.notify_all();
    cv.wait(lock, [] { return large_done; });
  }
  limit = value;
  ++sets;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes* a, const void*) {
  *a = cudaFuncAttributes{};
  a->sharedSizeBytes = kStatic;
  return cudaSuccess;
}
extern "C" cudaError_t cudaDeviceGetAttribute(int* value, enum cudaDeviceAttr attr, int) {
  if (attr != cudaDevAttrMaxSharedMemoryPerBlockOptin) return cudaErrorInvalidValue;
  *value = kOptin;
  return cudaSuccess;
}

static void kernel(int) {}

int main() {
  static std::atomic<int> granted[dsa::kMaxDevices];
  cudaError_t a, b;
  std::thread ta([&] {
    is_small = true;
    a = dsa::grant_smem(kernel, kSmall, 0, granted);
  });
  std::thread tb([&] {
    {
      std::unique_lock<std::mutex> lock(mu);
      cv.wait(lock, [] { return small_inside; });
    }
    b = dsa::grant_smem(kernel, kLarge, 0, granted);
    std::lock_guard<std::mutex> lock(mu);
    large_done = true;
    cv.notify_all();
  });
  ta.join();
  tb.join();
  const int before = sets;
  const cudaError_t c = dsa::grant_smem(kernel, kLarge, 0, granted);
  const cudaError_t d = dsa::grant_smem(kernel, kSmall, 0, granted, true);
  const cudaError_t too_much = dsa::grant_smem(kernel, kOptin, 0, granted);
  std::printf("%d %d %d %d %d %d %d %d\n", (int)a, (int)b, (int)c, (int)d, limit >= kLarge, limit + kStatic <= kOptin,
              sets - before, (int)(too_much != cudaSuccess));
  return 0;
}
"""


def test_the_larger_need_survives(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src = tmp_path / "grant.cpp"
    src.write_text(SOURCE)
    exe = tmp_path / "grant"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "long_context_05_b200", "csrc"), "-I", CUDA, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60)
    a, b, c, d, enough, within, later, refused = map(int, r.stdout.split())
    assert (a, b, c, d) == (0, 0, 0, 0)
    assert enough and within
    assert later <= 1                                  # asked once, not by every call
    assert refused
