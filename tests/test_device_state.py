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


def test_every_device_has_its_own_word(tmp_path):
    # a kernel that runs on one device must not be given another device's memory, however many threads ask first; what
    # cannot be made whole is asked for again by the next caller
    _run(tmp_path, r"""
#include <set>
#include <vector>
struct Piece { int dev, value; };
static std::mutex m;
static std::set<Piece*> pieces;
static int fail_malloc = 0, fail_memset = 0, errors = 0;
extern "C" cudaError_t cudaMalloc(void** p, size_t n) {
  std::lock_guard<std::mutex> lk(m);
  if (fail_malloc && fail_malloc--) { ++errors; return cudaErrorMemoryAllocation; }
  need(n == sizeof(int), "size");
  Piece* x = new Piece{t_dev, 77};
  pieces.insert(x);
  *p = x;
  return cudaSuccess;
}
extern "C" cudaError_t cudaMemset(void* p, int v, size_t n) {
  std::lock_guard<std::mutex> lk(m);
  if (fail_memset && fail_memset--) { ++errors; return cudaErrorInvalidValue; }
  need(v == 0 && n == sizeof(int), "cleared");
  static_cast<Piece*>(p)->value = 0;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFree(void* p) {
  std::lock_guard<std::mutex> lk(m);
  need(pieces.erase(static_cast<Piece*>(p)) == 1, "freed twice");
  return cudaSuccess;
}
extern "C" cudaError_t cudaGetLastError() { errors = 0; return cudaSuccess; }
int main() {
  static DeviceWord word;
  fail_malloc = fail_memset = 1;
  need(word.get() == nullptr && errors == 0 && pieces.empty(), "no memory");
  need(word.get() == nullptr && errors == 0 && pieces.empty(), "not cleared");
  std::vector<std::thread> threads;
  std::vector<int*> got(32);
  for (int i = 0; i < 32; ++i)
    threads.emplace_back([&got, i] { t_dev = i % 2 ? 5 : 0; got[i] = word.get(); });
  for (auto& t : threads) t.join();
  for (int i = 0; i < 32; ++i) {
    const Piece* p = reinterpret_cast<const Piece*>(got[i]);
    need(p && p->dev == (i % 2 ? 5 : 0) && p->value == 0 && got[i] == got[i % 2], "this device's word");
  }
  need(pieces.size() == 2, "one per device");
  t_dev = 64;
  need(word.get() == nullptr, "device past the table");
}
""")


def test_the_library_takes_its_error_word_by_device():
    # the per-step entries have no word of their own beside it
    import re
    from decoder_only_transformer_gpt_gb300 import build
    text = open(os.path.join(build.CSRC, "gptk.cu")).read()
    assert re.search(r"DeviceWord g_err;", text) and "cudaMalloc(&g_err" not in text
