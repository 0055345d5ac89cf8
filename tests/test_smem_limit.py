"""The shared-memory limit of a kernel under calls from two host threads. No GPU is used: the CUDA
calls of csrc/lq_smem.cu are stand-ins that record the limit."""
import ctypes
import os
import subprocess
import threading
import time

import fractional_bit_weight_b200 as lq
from fractional_bit_weight_b200 import build as lqbuild

HARNESS = r"""
#include <chrono>
#include <condition_variable>
#include <mutex>
#include "SOURCE"

static std::mutex m;
static std::condition_variable cv;
static int limit = 48 * 1024, sets = 0;

// The first call sets its limit and returns only when a second one has set another (or half a
// second later, if none can).
extern "C" cudaError_t cudaGetDevice(int* dev) { *dev = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
  std::unique_lock<std::mutex> held(m);
  limit = bytes;
  if (++sets == 1)
    cv.wait_for(held, std::chrono::milliseconds(500), [] { return sets > 1; });
  else
    cv.notify_all();
  return cudaSuccess;
}

static int cache[64];
extern "C" int ensure(int bytes) { return (int)lq::ensure_smem(nullptr, bytes, cache); }
extern "C" int limit_set() { return limit; }
extern "C" int first_is_in() { std::lock_guard<std::mutex> held(m); return sets > 0; }
"""


def test_two_threads_leave_the_larger_limit(tmp_path):
    source = os.path.join(lqbuild.CSRC, "lq_smem.cu")
    harness = tmp_path / "harness.cpp"
    harness.write_text(HARNESS.replace("SOURCE", source))
    out = tmp_path / "harness.so"
    subprocess.run([os.environ.get("NVCC", "nvcc"), "-x", "c++", "-std=c++17", "-shared", "-cudart",
                    "none", "-Xcompiler", "-fPIC", "-Xlinker", "-Bsymbolic",
                    "-I", lqbuild.CSRC, "-I", lqbuild.INCLUDE, "-o", str(out), str(harness)],
                   check=True)
    h = ctypes.CDLL(str(out))
    large, small = 230 * 1024, 150 * 1024
    first = threading.Thread(target=h.ensure, args=(large,))
    first.start()
    deadline = time.monotonic() + 30
    while not h.first_is_in() and time.monotonic() < deadline:
        time.sleep(0.001)
    assert h.first_is_in()
    assert h.ensure(small) == lq.LQ_OK      # from this thread, while the first call is under way
    first.join()
    assert h.ensure(large) == lq.LQ_OK
    assert h.limit_set() >= large
