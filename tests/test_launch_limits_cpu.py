"""The kernels' shared-memory limits under calls from several threads: host code
alone, with the CUDA calls behind it replaced."""
import shutil
import subprocess

import pytest

import structured_sparse_state_b200.build as build

SOURCE = r"""
#include <cuda_runtime.h>
#include <stdio.h>
#include <atomic>
#include <chrono>
#include <thread>
#include <vector>
static std::atomic<int> limit;      // what the kernel's last call left
static cudaError_t fake_get(int *dev) { *dev = 0; return cudaSuccess; }
static cudaError_t fake_set(const void *, cudaFuncAttribute, int bytes) {
    std::this_thread::sleep_for(std::chrono::microseconds(bytes % 7 * 50));
    limit = bytes;
    std::this_thread::sleep_for(std::chrono::microseconds(bytes % 5 * 50));
    return cudaSuccess;
}
#define cudaGetDevice fake_get
#define cudaFuncSetAttribute fake_set
#include "launch.cuh"
int main() {
    int bad = 0;
    for (int round = 0; round < 100; ++round) {
        std::atomic<int> set[pdssm::kLimitDevices] = {}, refused{0};
        limit = 0;
        std::vector<std::thread> threads;
        for (int i = 0; i < 8; ++i)
            threads.emplace_back([&, i] {
                const int bytes = 1000 + 37 * ((i * 5 + round * 3) % 8);
                if (pdssm::allow_smem(nullptr, bytes, set) != cudaSuccess || limit < bytes) ++refused;
            });
        for (auto &t : threads) t.join();
        bad += refused > 0 || limit != 1000 + 37 * 7;
    }
    printf("%d\n", bad);
    return bad != 0;
}
"""


@pytest.mark.skipif(not shutil.which(build._nvcc()), reason="needs nvcc")
def test_a_limit_is_never_lowered_under_another_threads_launch(tmp_path):
    src, exe = tmp_path / "limits.cu", tmp_path / "limits"
    src.write_text(SOURCE)
    subprocess.check_call([build._nvcc(), "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a",
                           "-I" + build.CSRC, "-I" + build.INCLUDE, str(src), "-o", str(exe)])
    assert subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True).stdout.strip() == "0"
