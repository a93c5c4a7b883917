"""The launch helpers' caches over several devices and launch shapes, on the host:
the helpers are compiled against counting stand-ins for the runtime calls that
they make, so no device is needed."""
import os
import subprocess

import pytest

from nvfp4_quantization_precision_gb300 import build as fos_build

SOURCE = r'''
#include <cuda_runtime.h>
#include <cstdio>

static int g_dev = 0, g_set = 0, g_occ = 0;
static cudaError_t fake_device(int* d) { *d = g_dev; return cudaSuccess; }
static cudaError_t fake_set(const void*, cudaFuncAttribute, int) { ++g_set; return cudaSuccess; }
// occupancy by what was asked: the device, the threads and the shared memory
static cudaError_t fake_occ(int* n, const void*, int threads, size_t smem) {
    ++g_occ;
    *n = 1 + g_dev + threads / 64 + (int)(smem >> 14);
    return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_set
#define cudaOccupancyMaxActiveBlocksPerMultiprocessor fake_occ
#include "fos_launch.cuh"

int main() {
    const void* k = &g_dev;   // stands for a kernel's address
    const void* other = &g_set;
    auto want = [](int got, int n, const char* what) {
        if (got != n) { std::printf("%s: %d instead of %d\n", what, got, n); return 1; }
        return 0;
    };
    int bad = 0;
    fos::allow_smem(k, 65536);
    fos::allow_smem(k, 65536);
    bad += want(g_set, 1, "one kernel, one device");
    g_dev = 1;
    fos::allow_smem(k, 65536);
    bad += want(g_set, 2, "the same kernel on a second device");
    g_dev = 17;
    fos::allow_smem(k, 65536);
    bad += want(g_set, 3, "and on device 17");
    g_dev = 0;
    fos::allow_smem(k, 65536);
    bad += want(g_set, 3, "back on the first");
    fos::allow_smem(k, 98304);
    fos::allow_smem(other, 65536);
    bad += want(g_set, 5, "more bytes; another kernel");
    fos::allow_smem(other, 1024);
    bad += want(g_set, 5, "below the default limit");
    for (int dev : {0, 1, 17})
        for (int threads : {256, 512})
            for (size_t smem : {size_t(0), size_t(65536)})
                for (int twice = 0; twice < 2; ++twice) {
                    g_dev = dev;
                    bad += want(fos::resident_ctas(k, smem, threads), 1 + dev + threads / 64 + (int)(smem >> 14),
                                "resident CTAs");
                }
    bad += want(g_occ, 12, "occupancy queries");
    return bad;
}
'''


@pytest.fixture(scope="module")
def nvcc():
    return fos_build._nvcc()


def test_attributes_and_occupancies_are_per_device(nvcc, tmp_path):
    src = tmp_path / "caches.cu"
    src.write_text(SOURCE)
    exe = tmp_path / "caches"
    r = subprocess.run([nvcc, *fos_build.NVFLAGS, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=dict(os.environ))
    assert r.returncode == 0, r.stdout


def test_no_cache_by_kernel_alone():
    """Every cache of the launchers is keyed by LaunchKey (or by the device), and
    function attributes are set by the one helper that knows the device."""
    for f in sorted(os.listdir(fos_build.CSRC)):
        text = open(os.path.join(fos_build.CSRC, f)).read()
        assert "cudaFuncSetAttribute" not in text or f == "fos_launch.cuh", f
        for line in text.splitlines():
            if "unordered_map<" in line:
                assert "unordered_map<LaunchKey" in line or "unordered_map<int," in line, (f, line)
