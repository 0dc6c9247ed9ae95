"""Host-side state of the fp8 launchers against a stand-in of the driver's calls, without a
GPU: host threads that meet inside a first call."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routed_expert_decode_gb300", "csrc")

SOURCE = r'''
#include <cstdio>
#include <thread>
#include <vector>
#include "fp8_host.h"

static int g_device, g_calls, g_value;          // the driver's state: the kernel's limit
static cudaError_t g_answer = cudaSuccess;
static void (*g_meanwhile)();                   // another thread's call, inside this one

extern "C" cudaError_t cudaGetDevice(int *d) { *d = g_device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int v) {
  ++g_calls;
  if (g_answer != cudaSuccess) return g_answer;
  if (auto f = g_meanwhile) { g_meanwhile = nullptr; g_value = v; f(); }
  else g_value = v;
  return cudaSuccess;
}
static void kernel(int) {}
static std::atomic<bool> done[moe::kMaxDevices];
static cudaError_t call() { return moe::allow_smem(kernel, done); }

#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
  const int all = (int)moe::kSmemLimit;
  // a failed call is asked again
  g_answer = cudaErrorInvalidValue;
  CHECK(call() == cudaErrorInvalidValue && call() == cudaErrorInvalidValue && g_calls == 2);
  g_answer = cudaSuccess;
  // a second thread's first call falls between this one's and its note of it: the
  // limit that stays is enough for any call after both
  g_meanwhile = [] { call(); };
  CHECK(call() == cudaSuccess && g_calls == 4 && g_value == all);
  g_value = -1;
  CHECK(call() == cudaSuccess && g_calls == 4 && g_value == -1);  // looked up no more
  // every device is asked once; one past the table each time
  g_device = 1;
  CHECK(call() == cudaSuccess && call() == cudaSuccess && g_calls == 5 && g_value == all);
  g_device = moe::kMaxDevices;
  CHECK(moe::device_here() == -1 && call() == cudaSuccess && call() == cudaSuccess && g_calls == 7);
  std::puts("ok");
  return 0;
}
'''


def test_shared_memory_limit_of_racing_calls(tmp_path):
    include = "/usr/local/cuda/include"
    if not os.path.exists(os.path.join(include, "cuda_runtime.h")):
        pytest.skip("no CUDA headers")
    src, exe = tmp_path / "host.cpp", tmp_path / "host"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", include, "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
