"""The launchers' per-device records (csrc/device_info.cpp) under threads: built
with ThreadSanitizer against a fake of the three CUDA calls it makes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "pagedattention_paged_kv_pa_b200", "csrc")

# devices 0 .. 3 have 100 + device SMs, device 70 is past the records, -1 fails
MAIN = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "serve_ops.h"

static thread_local int current = 0;
static std::atomic<int> attributes_set{0};
extern "C" cudaError_t cudaGetDevice(int* d) {
  *d = current;
  return current < 0 ? cudaErrorNoDevice : cudaSuccess;
}
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d) {
  *v = 100 + d;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) {
  ++attributes_set;
  return cudaSuccess;
}

int main() {
  std::atomic<unsigned long long> done{0};
  std::atomic<int> wrong{0};
  std::vector<std::thread> ts;
  for (int t = 0; t < 8; ++t)
    ts.emplace_back([&, t] {
      for (int i = 0; i < 2000; ++i) {
        current = (t + i) % 4;
        wrong += pa::device_sms() != 100 + current;
        wrong += pa::allow_smem(&done, 1000, done) != cudaSuccess;
      }
      current = 70;
      wrong += pa::device_sms() != 148;
      current = -1;
      wrong += pa::device_sms() != 148;
      wrong += pa::allow_smem(&done, 1000, done) != cudaErrorNoDevice;
    });
  for (auto& t : ts) t.join();
  // once a device, or once a thread that asked before the first was done
  if (attributes_set < 4 || attributes_set > 32 || done != 15) ++wrong;
  std::printf("wrong %d\n", wrong.load());
  return wrong != 0;
}
"""


def test_records_are_free_of_races(tmp_path):
    cxx = shutil.which("g++")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if cxx is None or not os.path.isdir(cuda):
        pytest.skip("no g++ or CUDA headers")
    (tmp_path / "probe.cpp").write_text("int main() {}\n")
    flags = [cxx, "-std=c++17", "-g", "-O1", "-fsanitize=thread", "-pthread"]
    probe = str(tmp_path / "probe")
    if subprocess.run(flags + ["-o", probe, str(tmp_path / "probe.cpp")],
                      capture_output=True).returncode or \
            subprocess.run([probe], capture_output=True).returncode:
        pytest.skip("ThreadSanitizer does not run here")
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "device_info")
    src = os.path.join(CSRC, "device_info.cpp")
    r = subprocess.run(flags + ["-I", cuda, "-I", CSRC, "-o", exe, str(tmp_path / "main.cpp"), src],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "data race" not in r.stderr, r.stdout + r.stderr[:4000]
