"""What the library keeps per device, from several host threads and on several devices: csrc/device_state.h compiled
against a runtime of the test's own (two devices, no GPU)."""
import os
import shutil
import subprocess

import pytest

FAKE = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <thread>
#include "device_state.h"
using namespace gptgb;
static void need(bool ok, const char* what) { if (!ok) { std::printf("%s\n", what); std::exit(1); } }
static thread_local int t_dev = 0;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = t_dev; return cudaSuccess; }
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d) { *v = 100 + d; return cudaSuccess; }
"""


def _run(tmp_path, body):
    from decoder_only_transformer_gpt_gb300 import build
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(FAKE + body)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, "-I", include, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_limit_never_falls_behind_a_larger_one(tmp_path):
    # two threads ask for 100 and 200 bytes at once. The runtime holds the first until the second has asked too (or a
    # while has passed), and the second's answer back until the first is through: what is recorded has to be what is set.
    _run(tmp_path, r"""
static std::mutex m;
static std::condition_variable cv;
static int asked = 0, set_to = 0;
static bool first_through = false;
static void kernel() {}
extern "C" cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int v) {
  need(f == reinterpret_cast<const void*>(&kernel), "kernel");
  std::unique_lock<std::mutex> lk(m);
  ++asked;
  cv.notify_all();
  if (v == 100) {
    cv.wait_for(lk, std::chrono::milliseconds(500), [] { return asked >= 2; });
    cv.wait_for(lk, std::chrono::milliseconds(100), [] { return set_to == 200; });
    set_to = v;
  } else {
    set_to = v;
    cv.notify_all();
    cv.wait_for(lk, std::chrono::milliseconds(500), [] { return first_through; });
  }
  return cudaSuccess;
}
int main() {
  static SmemLimit limit;
  std::thread a([] {
    need(limit.raise(&kernel, 0, 100) == cudaSuccess, "100");
    std::lock_guard<std::mutex> lk(m);
    first_through = true;
    cv.notify_all();
  });
  {
    std::unique_lock<std::mutex> lk(m);
    cv.wait(lk, [] { return asked >= 1; });
  }
  std::thread b([] { need(limit.raise(&kernel, 0, 200) == cudaSuccess, "200"); });
  a.join();
  b.join();
  need(limit.bytes[0] == 200 && set_to == 200, "recorded, but not set");
  const int before = asked;
  need(limit.raise(&kernel, 0, 150) == cudaSuccess && set_to == 200 && asked == before, "150 asks for nothing");
  need(limit.raise(&kernel, 1, 150) == cudaSuccess && asked == before + 1, "each device by itself");
}
""")


def test_sm_counts_by_device(tmp_path):
    _run(tmp_path, r"""
int main() {
  for (int d : {0, 1, 0, 63}) {
    int dev = -1, n = 0;
    t_dev = d;
    need(device_sms(&dev, &n) == cudaSuccess && dev == d && n == 100 + d, "count");
  }
  int dev, n;
  t_dev = 64;
  need(device_sms(&dev, &n) == cudaErrorInvalidDevice, "device past the table");
}
""")
