"""No C++ exception leaves the C entry points' host code: where memory runs out
there, nothing is thrown. A host program with stand-ins for the two CUDA calls
and an operator new that fails."""

import os
import shutil
import subprocess

import pytest

import paged_gqa_decode_reshape_gb300.build as pgb

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include "subset.h"

static bool no_memory = false;
static int set_calls = 0, device = 0;
void *operator new(std::size_t n) {
    if (no_memory) throw std::bad_alloc();
    return std::malloc(n);
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
extern "C" cudaError_t cudaGetDevice(int *dev) { *dev = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { ++set_calls; return cudaSuccess; }

int main() {
    char kernels[100];
    no_memory = true;
    try {
        for (int turn = 0; turn < 2; ++turn)
            for (device = 0; device < 3; ++device)
                for (int k = 0; k < 20; ++k)
                    if (pa::smem_once(kernels + k, 1000) != cudaSuccess) return 1;
        if (set_calls != 60) return 2;  // once per device and kernel
        device = 70;                    // a device or a kernel too many is set at every call
        for (int k = 0; k < 100; ++k)
            if (pa::smem_once(kernels + k, 1000) != cudaSuccess) return 3;
        device = 1;
        for (int k = 0; k < 100; ++k)
            if (pa::smem_once(kernels + k, 1000) != cudaSuccess) return 4;
    } catch (...) {
        return 5;
    }
    std::puts("ok");
}
"""


def test_kernel_attributes_are_set_without_memory(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(pgb.nvcc()))), "include")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-I", pgb.CSRC, "-I", cuda, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert (r.returncode, r.stdout.strip()) == (0, "ok")
