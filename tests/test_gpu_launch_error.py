"""A launch that the runtime refuses is reported once: by its return value, not
also as the last error that other code's next check would find."""
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include <cstdio>
#include "launch.cuh"

__global__ void put(int* word, int v) {
    fp8ll::await_dependency();
    *word = v;
}

int main() {
    int* word = nullptr;
    if (cudaMalloc(&word, sizeof(int)) != cudaSuccess) return 1;
    // no blocks: refused on the host, nothing is launched
    if (fp8ll::launch_dependent(put, 0u, 32u, 0, static_cast<cudaStream_t>(nullptr), word, 1) == cudaSuccess) return 2;
    if (cudaPeekAtLastError() != cudaSuccess) return 3;
    if (fp8ll::launch_dependent(put, 1u, 1u, 0, static_cast<cudaStream_t>(nullptr), word, 7) != cudaSuccess) return 4;
    int got = 0;
    if (cudaMemcpy(&got, word, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess || got != 7) return 5;
    return cudaFree(word) == cudaSuccess ? 0 : 6;
}
"""


def test_refused_launch_leaves_no_error_behind(tmp_path):
    from fp8_linear_layer_gb300 import build
    src, exe = tmp_path / "refused.cu", tmp_path / "refused"
    src.write_text(PROGRAM)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)], timeout=120).returncode == 0
