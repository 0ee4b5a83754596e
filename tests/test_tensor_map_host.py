"""csrc/tensor_map.cu from several threads (CPU only): each family of products looks the
driver's encoder up in its first call, under a lock of its own, so that first calls of two
families may do it at once; and the encoder wants a context, which a thread that has not
worked on the device yet has not got.  Built as plain C++ against a stand-in for the driver,
under ThreadSanitizer."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_finalize_rmsnorm_gb300", "csrc")

HARNESS = r"""
#include <atomic>
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>

#include "tensor_map.h"

static std::atomic<int> lookups{0}, maps{0};
static thread_local int device = 0;        // the thread's, as the runtime counts
static thread_local int context = -1;      // of a device, once it is set

extern "C" cudaError_t cudaGetDevice(int *d) { return *d = device, cudaSuccess; }
extern "C" cudaError_t cudaSetDevice(int d) { return device = context = d, cudaSuccess; }

static CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                       const cuuint64_t *, const cuuint32_t *box, const cuuint32_t *,
                       CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                       CUtensorMapFloatOOBfill) {
    if (context != device) return CUDA_ERROR_INVALID_CONTEXT;
    maps.fetch_add(1, std::memory_order_relaxed);
    return box[0] == 64 && box[1] == 32 ? CUDA_SUCCESS : CUDA_ERROR_INVALID_VALUE;
}

// fails at first, as where there is no driver yet
extern "C" cudaError_t cudaGetDriverEntryPointByVersion(const char *name, void **fn, unsigned,
                                                        unsigned long long,
                                                        cudaDriverEntryPointQueryResult *found) {
    if (std::strcmp(name, "cuTensorMapEncodeTiled") != 0) return cudaErrorInvalidValue;
    if (lookups.fetch_add(1, std::memory_order_relaxed) == 0) return cudaErrorInsufficientDriver;
    *fn = reinterpret_cast<void *>(&encode);
    *found = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

int main() {
    if (mf::find_encoder() != cudaErrorInsufficientDriver) return 2;
    std::atomic<int> ready{0};
    std::atomic<int> wrong{0};
    std::vector<std::thread> threads;
    constexpr int kThreads = 4;
    for (int i = 0; i < kThreads; ++i)
        threads.emplace_back([&, i] {
            device = i % 2;  // of a device that another thread works on, or not
            ready.fetch_add(1, std::memory_order_relaxed);
            while (ready.load(std::memory_order_relaxed) < kThreads) std::this_thread::yield();
            CUtensorMap m;
            if (mf::find_encoder() != cudaSuccess ||
                !mf::encode_map(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, nullptr, 2, {64, 32, 1}, {64, 0},
                                64, 32) ||
                device != i % 2 || context != device ||
                mf::encode_map(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, nullptr, 2, {64, 32, 1}, {64, 0},
                               65, 32))
                wrong.fetch_add(1, std::memory_order_relaxed);
        });
    for (auto &t : threads) t.join();
    std::printf("%d\n", maps.load());
    return wrong.load() ? 3 : 0;
}
"""


def compiled(tmp_path, name, sources):
    out = str(tmp_path / name)
    p = subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fsanitize=thread", "-pthread",
                        f"-I{CSRC}", "-I/usr/local/cuda/include",
                        f"-I{os.path.join(ROOT, 'include')}", "-x", "c++", *sources, "-o", out],
                       capture_output=True, text=True)
    return out, p


def test_first_calls_from_several_threads(tmp_path):
    probe = tmp_path / "probe.cpp"
    probe.write_text("int main() { return 0; }\n")
    out, p = compiled(tmp_path, "probe", [str(probe)])
    if p.returncode != 0 or subprocess.run([out], capture_output=True).returncode != 0:
        pytest.skip("no ThreadSanitizer here")
    harness = tmp_path / "harness.cpp"
    harness.write_text(HARNESS)
    out, p = compiled(tmp_path, "harness", [str(harness), os.path.join(CSRC, "tensor_map.cu")])
    assert p.returncode == 0, p.stderr
    for _ in range(5):
        r = subprocess.run([out], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr[:2000]
        assert r.stdout == "8\n"   # four maps, and four that are refused
