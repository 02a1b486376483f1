"""Several devices in one process, on the CPU: the library on a stand-in for the
CUDA runtime that knows, for each device, what its kernels were told."""
import subprocess
import sys

import pytest

from paged_kv_cache_xs_gb300 import build as xsbuild

# A launch fails where the current device has not been told of the kernel's shared memory.
RUNTIME = r"""
#include <cuda_runtime_api.h>
#include <stdlib.h>
static int dev, n_told, launches, told_dev[256], told_bytes[256], cluster, sms = 152, held[9] = {0, 152, 76, 0, 36, 0, 0, 0, 15};
static const void *told_fn[256];
extern "C" {
void fake_device(int d) { dev = d; }
void fake_held(int ctas, int n) { held[ctas] = n; }
int fake_launches(void) { return launches; }
int fake_cluster(void) { return cluster; }
cudaError_t cudaGetDevice(int *d) { *d = dev; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = sms; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute a, int v) {
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize && n_told < 256)
        told_fn[n_told] = f, told_dev[n_told] = dev, told_bytes[n_told++] = v;
    return cudaSuccess;
}
static int allowed(const void *f, size_t bytes) {
    if (bytes <= 48 << 10) return 1;
    for (int i = 0; i < n_told; ++i)
        if (told_fn[i] == f && told_dev[i] == dev && (size_t)told_bytes[i] >= bytes) return 1;
    return 0;
}
static int cluster_of(const cudaLaunchConfig_t *c) {
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return c->attrs[i].val.clusterDim.x;
    return 1;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *f, const cudaLaunchConfig_t *c) {
    if (!allowed(f, c->dynamicSmemBytes)) return cudaErrorInvalidValue;
    *n = held[cluster_of(c)];
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
    if (!allowed(f, c->dynamicSmemBytes)) return cudaErrorInvalidValue;
    cluster = cluster_of(c);
    ++launches;
    return cudaSuccess;
}
static int encode(void) { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *q) {
    *p = (void *)encode, *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
}
"""
CALLS = r"""
import ctypes, sys
from paged_kv_cache_xs_gb300 import ops
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ops.load()
A = 1 << 20          # never read: nothing runs
def prompt(T, start, Hq, Hkv, D, window=0):
    return lib.xs_paged_prefill_first(A, A, A, A, A, 4096, T, start, 4, window, Hq, Hkv, D, 16, 4096, 0.1, 1, None, None)
def causal(T, start, Hq, Hkv, D):
    return lib.xs_paged_prefill_tc(A, A, A, A, A, 4096, T, start, Hq, Hkv, D, 16, 4096, 0.1, 1, None, None)
def decode(name, B, Hq, Hkv, D, dtype, maxb=64):
    if name == "first":
        return lib.xs_paged_decode_first(A, A, Hq * D, A, A, A, maxb, A, None, 4, 100, B, Hq, Hkv, D, 16, 4096, 0.1, A, 1 << 40,
                                         dtype, None, None)
    return lib.xs_paged_decode_weights(A, A, None, A, Hq * D, A, A, A, maxb, A, None, B, Hq, Hkv, D, 16, 4096, 0.1, A, 1 << 40,
                                       dtype, None, None)
def evict(maxb):
    return lib.xs_kv_evict(A, 3, A, A, 1, 4096 * 2 * 4096, A, A, maxb, A, 3, None, 4, 8, 64, 80, 2, 128, 16, 4096, 1, A, A, None,
                           None)
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    xsbuild.build()
    d = tmp_path_factory.mktemp("runtime")
    (d / "runtime.cpp").write_text(RUNTIME)
    include = xsbuild.os.path.join(xsbuild.os.path.dirname(xsbuild.os.path.dirname(xsbuild.os.path.realpath(xsbuild.nvcc()))),
                                   "include")
    so = d / "runtime.so"
    subprocess.run(["g++", "-shared", "-fPIC", "-w", "-I", include, str(d / "runtime.cpp"), "-o", str(so)], check=True)

    def run(code):
        env = {**xsbuild.os.environ, "LD_PRELOAD": str(so), "PYTHONPATH": xsbuild.ROOT}
        r = subprocess.run([sys.executable, "-c", CALLS + code, str(so)], capture_output=True, text=True, env=env, cwd=xsbuild.ROOT)
        assert r.returncode == 0, r.stderr
        return r.stdout
    return run


def test_each_device_is_told_of_the_prompt_kernels_shared_memory(fake):
    fake("""
for dev in (0, 1, 5, 0, 70, 70, 1):
    fake.fake_device(dev)
    for D in (64, 128):
        for G in (1, 2, 4, 8):
            for T in (1, 300, 40000):
                assert prompt(T, 500, 8 * G, 8, D, 64) == 0, (dev, D, G, T)
                assert causal(T, 500, 8 * G, 8, D) == 0, (dev, D, G, T)
assert fake.fake_launches() == 7 * 2 * 4 * 3 * 2
""")


def test_each_device_is_told_of_the_other_bounded_kernels_shared_memory(fake):
    fake("""
for dev in (0, 1, 70, 0):
    fake.fake_device(dev)
    for D in (64, 128):
        for dtype in (0, 1):
            for B in (1, 10, 40, 400):
                assert decode("first", B, 8, 2, D, dtype) == 0 and decode("weights", B, 8, 2, D, dtype) == 0, (dev, D, dtype, B)
    assert evict(4) == 0 and evict(4096) == 0, dev
""")


def test_prompt_clusters_are_what_the_device_holds(fake):
    # 8 Q tiles of one query, their keys shared by the largest clusters that are held 8 at a time.
    fake("""
for dev, held, want in ((0, (76, 36, 15), 8), (1, (70, 30, 7), 4), (2, (60, 7, 8), 2), (3, (7, 20, 20), 1), (0, (0, 0, 0), 8)):
    fake.fake_device(dev)
    for i in range(3):
        fake.fake_held(2 << i, held[i])
    for D in (64, 128):
        assert prompt(1, 3000, 32, 8, D) == 0 and fake.fake_cluster() == want, (dev, D, fake.fake_cluster())
""")
