"""Host code that several threads share, against stand-ins for the CUDA runtime's calls (no GPU
needed)."""
import os
import subprocess

from expert_ffn_layer_router_b200 import build as lib_build

# Two threads ask for different sizes of one kernel.  The stand-in holds the smaller request back until
# the larger one has been granted, or for half a second if that one is not let in meanwhile.
RUNTIME = r"""
#include <atomic>
#include <chrono>
#include <thread>

std::atomic<int> limit{0}, large_done{0}, small_in{0};

extern "C" int cudaGetDevice(int* dev) { *dev = 0; return 0; }
extern "C" int cudaFuncSetAttribute(const void*, int, int bytes) {
    if (bytes == 1000) {
        small_in = 1;
        for (int i = 0; i < 500 && !large_done; ++i)
            std::this_thread::sleep_for(std::chrono::milliseconds(1));
    }
    limit = bytes;
    if (bytes == 2000) large_done = 1;
    return 0;
}
"""

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include "common.cuh"

extern std::atomic<int> limit, small_in;
static void kernel(int) {}
static std::atomic<int> allowed[64];

int main() {
    std::thread a([] { moe::allow_smem(kernel, allowed, 1000); });
    while (!small_in) std::this_thread::yield();
    std::thread b([] { moe::allow_smem(kernel, allowed, 2000); });
    a.join();
    b.join();
    moe::allow_smem(kernel, allowed, 1500);
    std::printf("%d %d\n", limit.load(), allowed[0].load());
    return 0;
}
"""


def test_shared_memory_limit_is_never_lowered(tmp_path):
    src, runtime, exe = tmp_path / "limit.cu", tmp_path / "runtime.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    runtime.write_text(RUNTIME)
    subprocess.run([lib_build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                    "--cudart", "shared", "-I", lib_build.CSRC, str(src), str(runtime), "-o", str(exe)],
                   check=True)
    # (the shared runtime's start-up symbols resolve there; the two calls above to the stand-ins)
    libs = os.path.join(os.path.dirname(os.path.dirname(lib_build.nvcc())), "lib64")
    env = {**os.environ, "LD_LIBRARY_PATH": libs + ":" + os.environ.get("LD_LIBRARY_PATH", "")}
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60,
                         env=env).stdout
    assert out.split() == ["2000", "2000"]
