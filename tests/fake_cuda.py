"""liber.so over a stand-in for the CUDA runtime: host memory, a current device that tests set, launches that do nothing and an
order of events that tests read.  For what the host side does around the GPU, without one."""

from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

SOURCE = r"""
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>
#define OUT __attribute__((visibility("default")))
OUT int fake_device, fake_pending, fake_pointer_device, fake_launches;
OUT void *fake_last_alloc;
OUT cudaError_t cudaGetDevice(int *d) { *d = fake_device; return cudaSuccess; }
OUT cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr a, int d) {
    (void)d;
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : 1 << 20;
    return cudaSuccess;
}
OUT cudaError_t cudaFuncSetAttribute(const void *f, enum cudaFuncAttribute a, int v) { (void)f, (void)a, (void)v; return cudaSuccess; }
OUT cudaError_t cudaMalloc(void **p, size_t n) {
    n = (n + 255) / 256 * 256;
    *p = fake_last_alloc = aligned_alloc(256, n);
    memset(*p, 0xEE, n);
    return cudaSuccess;
}
OUT cudaError_t cudaFree(void *p) { free(p); return cudaSuccess; }
// returns before the GPU has done it, as on device memory
OUT cudaError_t cudaMemset(void *p, int v, size_t n) { memset(p, v, n); fake_pending = 1; return cudaSuccess; }
OUT cudaError_t cudaMemcpy(void *d, const void *s, size_t n, enum cudaMemcpyKind k) { (void)k; memcpy(d, s, n); return cudaSuccess; }
OUT cudaError_t cudaMemcpyAsync(void *d, const void *s, size_t n, enum cudaMemcpyKind k, cudaStream_t t) {
    (void)k, (void)t;
    memcpy(d, s, n);
    return cudaSuccess;
}
OUT cudaError_t cudaMemsetAsync(void *p, int v, size_t n, cudaStream_t t) { (void)t; memset(p, v, n); return cudaSuccess; }
OUT cudaError_t cudaStreamCreateWithFlags(cudaStream_t *t, unsigned f) { (void)f; *t = (cudaStream_t)1; return cudaSuccess; }
OUT cudaError_t cudaStreamDestroy(cudaStream_t t) { (void)t; return cudaSuccess; }
OUT cudaError_t cudaStreamSynchronize(cudaStream_t t) { (void)t; return cudaSuccess; }
OUT cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *f, int b, size_t m, unsigned x) {
    (void)f, (void)b, (void)m, (void)x;
    *n = 1;
    return cudaSuccess;
}
OUT cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes *a, const void *f) { (void)f; memset(a, 0, sizeof *a); return cudaSuccess; }
OUT cudaError_t cudaDeviceSynchronize(void) { fake_pending = 0; return cudaSuccess; }
OUT cudaError_t cudaPointerGetAttributes(struct cudaPointerAttributes *a, const void *p) {
    memset(a, 0, sizeof *a);
    a->type = p ? cudaMemoryTypeDevice : cudaMemoryTypeUnregistered;
    a->device = p ? fake_pointer_device : -2;
    return cudaSuccess;
}
OUT cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) { *k = (cudaKernel_t)f; return cudaSuccess; }
OUT cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 g, dim3 b, void **args, size_t n, cudaStream_t s) {
    (void)k, (void)g, (void)b, (void)args, (void)n, (void)s;
    ++fake_launches;
    return cudaSuccess;
}
OUT cudaError_t cudaGetLastError(void) { return cudaSuccess; }
"""

PRELUDE = """
import ctypes
from block_quantized_token_gb300 import er
fake = ctypes.CDLL(None)
def word(name):
    return ctypes.c_int.in_dll(fake, name)
def refused(f, *a):
    try:
        f(*a)
    except er.ErError as e:
        return e.status
    return er.ER_OK
cfg = er.er_pages_config(2, 10, 32, 3, 64, er.ER_Q4_0)
pool = (ctypes.c_uint8 * (er.er_pages_pool_bytes(cfg) + 256))()
pool_ptr = (ctypes.addressof(pool) + 255) // 256 * 256
ints = (ctypes.c_int32 * 4096)()
at = ctypes.addressof(ints)
"""


def run(tmp_path, script: str) -> None:
    """Runs `script` (after PRELUDE) in a process whose liber.so finds the stand-in first."""
    from block_quantized_token_gb300 import build
    build.build()
    src, lib = os.path.join(tmp_path, "fake.c"), os.path.join(tmp_path, "fake.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-w", "-I", os.path.join(CUDA, "include"), "-o", lib, src], check=True)
    env = dict(os.environ, LD_PRELOAD=lib, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", PRELUDE + script], env=env, cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
