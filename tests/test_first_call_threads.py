"""The chunk-attention launches look the driver's tensor-map encoder up once a process.  Threads
whose first calls overlap must all get it: compiled from the kernels' own header with a lookup
that takes its time."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cuda_runtime.h>
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
static std::atomic<int> lookups{0};
static cudaError_t slow_lookup(const char *, void **p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *q) {
    lookups++;
    std::this_thread::sleep_for(std::chrono::milliseconds(200));
    *p = reinterpret_cast<void *>(&slow_lookup);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
#define cudaGetDriverEntryPointByVersion slow_lookup
#include "extend_common.cuh"
int main() {
    std::atomic<int> missing{0};
    std::thread t[8];
    for (auto &x : t) x = std::thread([&] { missing += nvfp4kv::encode_fn() == nullptr; });
    for (auto &x : t) x.join();
    std::printf("%d missing, %d lookups\n", missing.load(), lookups.load());
    return missing.load() != 0 || lookups.load() != 1;
}
"""


def test_threads_whose_first_calls_overlap_all_get_the_encoder(tmp_path):
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    nvcc = cand if os.path.exists(cand) else shutil.which("nvcc")
    if not nvcc:
        pytest.skip("nvcc not available")
    (tmp_path / "t.cu").write_text(SOURCE)
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "nvfp4_quantised_paged_gb300", "csrc"), str(tmp_path / "t.cu"), "-o",
                        str(tmp_path / "t")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
