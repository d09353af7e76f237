"""How many clusters fit on the device is asked once and remembered; a query that
fails is not.  Compiled with nvcc against a runtime of the test's own whose calls
fail when told to (no GPU needed)."""
import os
import subprocess

from semi_structured_sparse_diag_b200 import build

PROGRAM = r"""
#include "nm_gemm.cuh"
#include <stdio.h>

static int fail_occupancy = 0, fail_attribute = 0, asked = 0;

#ifndef __CUDA_ARCH__  // the device pass has its own
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 148; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) {
    return fail_attribute ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *q) {
    ++asked;
    *n = q->gridDim.x / q->attrs[0].val.clusterDim.x;
    return fail_occupancy ? cudaErrorUnknown : cudaSuccess;
}
void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
char __cudaInitModule(void **) { return 0; }
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, struct CUstream_st *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t cudaLaunchKernel(const void *, dim3, dim3, void **, size_t, cudaStream_t) { return cudaErrorUnknown; }
}
#endif

__global__ void kernel() {}

int main() {
    auto ask = [](int pairs) { return static_cast<long>(nm::resident_clusters_of<kernel>(pairs, 128, 1024)); };
    fail_occupancy = 1;
    printf("%ld %ld ", ask(1), ask(8));
    fail_occupancy = 0;
    fail_attribute = 1;  // the shared memory is settled: the wide clusters' permission fails
    printf("%ld ", ask(8));
    fail_attribute = 0;
    printf("%ld %ld ", ask(1), ask(8));
    const int once = asked;
    fail_occupancy = fail_attribute = 1;  // remembered: not asked again
    printf("%ld %ld %d %ld\n", ask(1), ask(8), asked - once, ask(9));
    return 0;
}
"""


def test_a_failed_query_is_not_remembered(tmp_path):
    src, exe = tmp_path / "query.cu", tmp_path / "query"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-cudart", "none", "--expt-relaxed-constexpr", "-I", build.CSRC,
                    "-I", os.path.join(build.HERE, "..", "include"), str(src), "-o", str(exe)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert out.split() == ["-1", "-1", "-1", "74", "9", "74", "9", "0", "-1"]
