"""The library's record of the kernels' shared-memory limits, between threads:
its source compiled against a stand-in for the CUDA runtime, whose calls meet in
the order that loses an unlocked record (the smaller limit is set last, the
larger one recorded last)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "bit_expert_gemv_b200", "csrc", "smem.cu")
CUDA = "/usr/local/cuda/include"

PROGRAM = r"""
#include <cuda_runtime_api.h>
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
namespace gale { int ensure_smem(const void* kernel, int bytes); }
static std::atomic<int> limit{0}, calls{0};
static void sleep_ms(int n) { std::this_thread::sleep_for(std::chrono::milliseconds(n)); }
extern "C" cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, enum cudaFuncAttribute, int bytes) {
    ++calls;
    for (int i = 0; i < 300 && calls < 2; ++i) sleep_ms(1);      // the other thread's call, if it can come in
    if (bytes == 100) sleep_ms(50);
    limit = bytes;
    if (bytes == 200) sleep_ms(100);
    return cudaSuccess;
}
int main() {
    int kernel, others[40];
    std::thread small([&] { gale::ensure_smem(&kernel, 100); }), large([&] { gale::ensure_smem(&kernel, 200); });
    small.join();
    large.join();
    if (gale::ensure_smem(&kernel, 200) != 0 || limit != 200) return 1;
    if (gale::ensure_smem(&kernel, 150) != 0 || limit != 200) return 2;       // never lowered
    for (int i = 0; i < 40; ++i)                                              // every kernel has its own record
        if (gale::ensure_smem(&others[i], 300 + i) != 0 || limit != 300 + i) return 3;
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(CUDA), reason="no g++ or CUDA headers")
def test_limits_between_threads(tmp_path):
    main, exe = tmp_path / "main.cpp", tmp_path / "main"
    main.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I", CUDA, str(main), "-x", "c++",
                    SOURCE, "-o", str(exe), "-lpthread"], check=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0
