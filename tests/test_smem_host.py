"""The limit of a kernel's dynamic shared memory with several host threads (no GPU: the two CUDA calls are stand-ins)."""
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The larger request's thread is held inside the CUDA call until the smaller one's has gone through it too (or 300 ms)
SOURCE = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "smem.cuh"

static std::atomic<int> attribute{0}, inside{0}, others{0};

cudaError_t cudaGetDevice(int *dev) { *dev = 0; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int bytes)
{
    attribute = bytes;
    if (bytes == 100000) {
        inside = 1;
        for (int i = 0; i < 300 && !others; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
    }
    return cudaSuccess;
}
static void kernel(int) {}

int main()
{
    static ssd::SmemLimit limit;
    bool a = false, b = false;
    std::thread large([&] { a = ssd::allow_smem(kernel, 100000, limit); });
    while (!inside) std::this_thread::yield();
    std::thread small([&] { b = ssd::allow_smem(kernel, 60000, limit); others = 1; });
    large.join();
    small.join();
    const int both = attribute;
    const bool again = ssd::allow_smem(kernel, 90000, limit);
    const int kept = attribute;
    const bool more = ssd::allow_smem(kernel, 200000, limit) && ssd::allow_smem(kernel, 70000, limit);
    std::printf("%d %d %d %d: %d %d %d\n", a, b, again, more, both, kept, attribute.load());
    return a && b && again && more && both == 100000 && kept == 100000 && attribute == 200000 ? 0 : 1;
}
"""


def test_a_limit_is_never_lowered(tmp_path):
    nvcc = shutil.which("nvcc")
    assert nvcc, "nvcc builds the library: it has to be on the path"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-pthread", "-I", include, "-I", os.path.join(ROOT, "mamba_selective_state_causal_b200", "csrc"),
                           str(src), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
