"""CPU test of the host state that kernels keep per device: a small program over csrc/txl_once.h with a cudaGetDevice of
its own.  And no launch may go back to a flag per process: function attributes belong to one device."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "transformer_xl_relative_gb300", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

PROGRAM = r"""
#include "txl_once.h"
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>
static thread_local int device = 0;
static std::atomic<int> set_on[128];
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes)
{
    if (answer == cudaSuccess && bytes == 1000) ++set_on[device];
    return answer;
}
static void one() {}
static void two(int) {}
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main()
{
    txl::OncePerDevice once;
    auto ask = [&](int d) { device = d; return txl::allow_smem(once, 1000, one, two); };
    CHECK(ask(0) == cudaSuccess && ask(0) == cudaSuccess && set_on[0] == 2);       // both kernels, once
    CHECK(ask(1) == cudaSuccess && ask(1) == cudaSuccess && set_on[1] == 2);       // and on the second device
    CHECK(ask(63) == cudaSuccess && ask(63) == cudaSuccess && set_on[63] == 2);
    CHECK(ask(64) == cudaSuccess && ask(64) == cudaSuccess && set_on[64] == 4);    // not remembered
    answer = cudaErrorInvalidValue;
    CHECK(ask(0) == cudaSuccess && ask(2) == cudaErrorInvalidValue && set_on[2] == 0);
    answer = cudaSuccess;
    CHECK(ask(2) == cudaSuccess && set_on[2] == 2);                                // tried again
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&] { for (int d = 8; d < 40; ++d) if (ask(d) != cudaSuccess) std::abort(); });
    for (auto& t : threads) t.join();
    for (int d = 8; d < 40; ++d) {
        const int n = set_on[d];
        CHECK(n >= 2 && ask(d) == cudaSuccess && set_on[d] == n);
    }
    return 0;
}
"""


def test_once_per_device(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-I", os.path.join(CUDA, "include"), str(src),
                    "-o", str(exe)], check=True, timeout=120)
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert p.returncode == 0, p.stdout


def test_no_launch_keeps_a_flag_per_process():
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name), encoding="utf-8").read()
        assert not re.search(r"\bstatic\s+(std::atomic<)?bool\b", text), name
