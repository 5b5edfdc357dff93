"""A launch that fails in the middle of a call: the call says so, and leaves
nothing behind that the next one would go by.  The library's own objects run
over a stand-in for the CUDA runtime, on the host: its kernels do nothing, its
device memory is the host's, and the launch that a test names returns an error."""
import ctypes
import glob
import os
import shutil
import subprocess

import pytest

from continuous_linear_attention_gb300 import build

RUNTIME = r"""
#include <cstdlib>
#include <cstring>
#include <cstddef>
typedef int err;
static int launches = 0, failing = -1;
static void* last_alloc[8];
static int allocs = 0;
static err launch() { return launches++ == failing ? 2 : 0; }
extern "C" {
void fake_fail(int at) { launches = 0; failing = at; }
int fake_launches() { return launches; }
void* fake_alloc(int i) { return i < allocs ? last_alloc[i] : nullptr; }
void fake_reset() { allocs = 0; }
err cudaLaunchKernelExC(const void*, const void*, void**) { return launch(); }
err __cudaLaunchKernel(...) { return launch(); }
err __cudaGetKernel(void** k, const void* f) { *k = const_cast<void*>(f); return 0; }
unsigned __cudaPushCallConfiguration(...) { return 0; }
err __cudaPopCallConfiguration(...) { return 0; }
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(...) {}
void __cudaRegisterVar(...) {}
err cudaDeviceGetAttribute(int* v, int, int) { *v = 152; return 0; }
err cudaDeviceSynchronize() { return 0; }
err cudaEventRecord(void*, void*) { return 0; }
err cudaFree(void* p) { free(p); return 0; }
err cudaFreeAsync(void* p, void*) { free(p); return 0; }
err cudaFuncSetAttribute(const void*, int, int) { return 0; }
err cudaGetDevice(int* d) { *d = 0; return 0; }
err cudaSetDevice(int) { return 0; }
err cudaGetLastError() { return 0; }
const char* cudaGetErrorString(err) { return ""; }
static int encode(...) { return 0; }
err cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long, int* q) {
  *f = (void*)encode;
  *q = 0;
  return 0;
}
err cudaGetSymbolAddress(void**, const void*) { return 2; }
err cudaMalloc(void** p, size_t n) {
  *p = aligned_alloc(256, (n + 255) / 256 * 256);
  memset(*p, 0x5a, n);
  if (allocs < 8) last_alloc[allocs++] = *p;
  return 0;
}
err cudaMallocAsync(void** p, size_t n, void*) { return cudaMalloc(p, n); }
err cudaMemcpyAsync(void* d, const void* s, size_t n, int, void*) { memmove(d, s, n); return 0; }
err cudaMemset(void* p, int v, size_t n) { memset(p, v, n); return 0; }
err cudaMemsetAsync(void* p, int v, size_t n, void*) { memset(p, v, n); return 0; }
err cudaStreamIsCapturing(void*, int* s) { *s = 0; return 0; }
err cudaStreamSynchronize(void*) { return 0; }
}
"""
ERR_CUDA = -5


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    objects = sorted(glob.glob(os.path.join(build.BUILD_DIR, "*.cu.o")))
    if len(objects) != len(glob.glob(os.path.join(build.CSRC, "*.cu"))):
        build.build(force=True)
        objects = sorted(glob.glob(os.path.join(build.BUILD_DIR, "*.cu.o")))
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    where = tmp_path_factory.mktemp("fake")
    src, out = where / "runtime.cpp", where / "libfake.so"
    src.write_text(RUNTIME)
    # (-Bsymbolic: the calls stay in this library, whatever runtime the process has loaded)
    subprocess.run([cxx, "-shared", "-fPIC", "-O1", "-Wl,-Bsymbolic", "-Wl,-z,defs", "-o", str(out), str(src), *objects,
                    "-lpthread"], check=True, capture_output=True)
    lib = ctypes.CDLL(str(out))
    lib.fake_alloc.restype = ctypes.c_void_p
    P, I, L, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.gdn_win_pool_create.argtypes = [ctypes.POINTER(P)] + [I] * 7 + [S, P, S]
    lib.gdn_win_varlen_forward.argtypes = [P, I, P, P, P, L, L, L, I, P, P, P, ctypes.c_float, P, L, I, I, I, P]
    lib.gdn_state_pool_destroy.argtypes = [P]
    return lib


@pytest.mark.parametrize("N,T", [(1, 500), (4, 500), (300, 900)])
@pytest.mark.parametrize("act,d", [(1, 128), (1, 64), (1, 32), (0, 64)])
def test_windowed_attention(lib, N, T, act, d):
    """The prompts' form claims units from a counter and counts those it leaves;
    a kernel behind it sets both back, or, where that was not launched, the call."""
    pool, layer, blocks = ctypes.c_void_p(), 1, 8
    lib.fake_fail(-1)
    lib.fake_reset()
    assert lib.gdn_win_pool_create(ctypes.byref(pool), blocks, 2, 2, d, 64, 4, act, 0, None, 0) == 0
    # the pool's memory, then the work area: a header of 16 words and 8 for each block and 1, per layer
    words = 16 + 8 * blocks + 1
    header = ctypes.cast(lib.fake_alloc(1) + 4 * words * layer, ctypes.POINTER(ctypes.c_int32))
    assert list(header[:16]) == [0] * 16
    buf = (ctypes.c_char * (1 << 16))()
    at = (ctypes.addressof(buf) + 255) // 256 * 256

    def call():
        return lib.gdn_win_varlen_forward(pool, layer, at, at, at, 4 * d, 2 * d, 2 * d, 4, at, at, at, 1.0, at, 4 * d,
                                          T, N, 0, None)

    lib.fake_fail(-1)
    assert call() == 0
    n = lib.fake_launches()
    assert n >= 2
    for k in range(n):
        header[5], header[7] = 3, 9  # (as the kernels before the failing one leave them)
        lib.fake_fail(k)
        assert call() == ERR_CUDA, k
        assert lib.fake_launches() == k + 1
        if act == 1 and d >= 64 and k > (N > 256):  # behind the prompts' kernel
            assert (header[5], header[7]) == (0, 0), k
    lib.gdn_state_pool_destroy(pool)


def test_refused_scales_launch_nothing(lib):
    pool = ctypes.c_void_p()
    lib.fake_fail(-1)
    lib.fake_reset()
    assert lib.gdn_win_pool_create(ctypes.byref(pool), 8, 1, 2, 64, 64, 4, 1, 0, None, 0) == 0
    buf = (ctypes.c_char * (1 << 16))()
    at = (ctypes.addressof(buf) + 255) // 256 * 256

    def call(scale):
        lib.fake_fail(-1)
        status = lib.gdn_win_varlen_forward(pool, 0, at, at, at, 256, 128, 128, 4, at, at, at, scale, at, 256, 500, 4, 0,
                                            None)
        return status, lib.fake_launches() > 0

    for scale in (float("nan"), float("inf"), -float("inf"), 1.8e38, -3.4e38):
        assert call(scale) == (-3, False), scale
    for scale in (0.0, 1.0, -1.0, 2.0 ** 127, -2.0 ** 127, 1e-38):
        assert call(scale) == (0, True), scale
    lib.gdn_state_pool_destroy(pool)
