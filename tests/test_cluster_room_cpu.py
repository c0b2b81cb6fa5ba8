"""What launches in clusters remember of a device: the host code of kda_clusters.cuh built into a program whose CUDA calls are fakes
that count, answer by device, and fail."""
import os
import subprocess

import pytest

from kimi_delta_attention_chunk_gb300 import build as kbuild

FAKES = r"""
#include <stdio.h>

#include <cuda_runtime_api.h>

int device, asked, attributes;
cudaError_t answer = cudaSuccess;
static const int room[3] = {0, 40, 80};

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
    ++asked;
    if (answer == cudaSuccess) *n = room[device];
    return answer;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { ++attributes; return answer; }
cudaError_t cudaGetLastError() { printf("an error was cleared\n"); return answer; }
}
"""

PROGRAM = r"""
#include <stdio.h>

#include "kda_clusters.cuh"

extern int device, asked, attributes;
extern cudaError_t answer;
static void kernel(int) {}
static int failed;
#define CHECK(x) \
    if (!(x)) printf("line %d: %s\n", __LINE__, #x), failed = 1

static kda::ClusterRoom rooms;
static int size_of(int64_t groups, int T, cudaError_t* e) {
    int size = -1;
    *e = rooms.size_for(kernel, groups, T, 128, 256, 1 << 16, size);
    return size;
}

int main() {
    cudaError_t e;
    // each device its own answer, asked for once a size
    device = 1;
    CHECK(size_of(30, 16384, &e) == 8 && e == cudaSuccess && asked == 1);
    CHECK(size_of(30, 16384, &e) == 8 && asked == 1);
    CHECK(size_of(60, 16384, &e) == 1 && e == cudaSuccess && asked == 7);
    device = 2;
    CHECK(size_of(60, 16384, &e) == 8 && e == cudaSuccess && asked == 8);
    CHECK(size_of(60, 300, &e) == 3 && asked == 9);
    CHECK(size_of(60, 100, &e) == 1 && asked == 9);
    device = 1;
    CHECK(size_of(60, 16384, &e) == 1 && asked == 9);
    // no room at all is an answer too
    device = 0;
    CHECK(size_of(1, 16384, &e) == 1 && e == cudaSuccess && asked == 16);
    CHECK(size_of(1, 16384, &e) == 1 && asked == 16);
    // a failure reaches the caller and is not remembered
    kda::ClusterRoom* const fresh = new kda::ClusterRoom();
    int size;
    answer = cudaErrorInvalidValue;
    device = 2;
    CHECK(fresh->size_for(kernel, 60, 16384, 128, 256, 1 << 16, size) == cudaErrorInvalidValue);
    answer = cudaSuccess;
    CHECK(fresh->size_for(kernel, 60, 16384, 128, 256, 1 << 16, size) == cudaSuccess && size == 8);
    // devices beyond those that are kept are asked every time
    int n;
    asked = 0;
    for (int k = 0; k < 2; ++k) CHECK(fresh->of(kernel, 64, 8, 256, 1 << 16, n) == cudaSuccess && n == 80);
    CHECK(asked == 2);
    // shared memory: what a kernel declares counts, every device is asked once, a failure not at all
    std::atomic<uint64_t> done{0};
    CHECK(kda::allow_shared(kernel, 512, 24 * 1024, done) == cudaSuccess && attributes == 0);
    CHECK(kda::allow_shared(kernel, 40 * 1024, 20 * 1024, done) == cudaSuccess && attributes == 1);
    CHECK(kda::allow_shared(kernel, 40 * 1024, 20 * 1024, done) == cudaSuccess && attributes == 1);
    device = 1;
    answer = cudaErrorInvalidValue;
    CHECK(kda::allow_shared(kernel, 0, 50 * 1024, done) == cudaErrorInvalidValue && attributes == 2);
    answer = cudaSuccess;
    CHECK(kda::allow_shared(kernel, 0, 50 * 1024, done) == cudaSuccess && attributes == 3);
    CHECK(kda::allow_shared(kernel, 0, 50 * 1024, done) == cudaSuccess && attributes == 3);
    if (!failed) printf("all right\n");
    return failed;
}
"""


def test_rooms_and_marks_by_device(tmp_path):
    try:
        nvcc = kbuild.nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    source, fakes, program = tmp_path / "rooms.cu", tmp_path / "fakes.cpp", str(tmp_path / "rooms")
    source.write_text(PROGRAM)
    fakes.write_text(FAKES)
    flags = [f for f in kbuild.NVCC_FLAGS if f != "-lineinfo"]
    built = subprocess.run([nvcc, *kbuild.ARCH, *flags, "-cudart", "shared", "-I", kbuild.CSRC, str(source), str(fakes), "-o", program], capture_output=True, text=True)
    assert built.returncode == 0, built.stdout + built.stderr
    libs = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    run = subprocess.run([program], capture_output=True, text=True, timeout=60,
                         env={**os.environ, "LD_LIBRARY_PATH": libs + os.pathsep + os.environ.get("LD_LIBRARY_PATH", "")})
    assert run.returncode == 0 and run.stdout == "all right\n", run.stdout + run.stderr
