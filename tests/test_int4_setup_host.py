"""The INT4 decode's set-up of its kernels against a stand-in for the CUDA runtime: a call of it that fails does not leave a
half-made entry behind."""
import ctypes
import os
import shutil
import subprocess

import pytest

from paged_kv_cache_252_gb300 import build

RUNTIME = r"""
#include "decode_int4.cu"
namespace pkv {
int device_sm_count(int* sms) { *sms = 152; return 0; }
bool cache_desc_ok(const pkv_cache_desc*) { return true; }
uint32_t next_call_epoch() { return 1; }
int launch_overlapped(const void*, dim3, dim3, size_t, void*, void**) { return 0; }
DecodeInt4Kernel decode_int4_kernel_f16(int, int) { return {"a", 128, 1000}; }
DecodeInt4Kernel decode_int4_kernel_bf16(int, int) { return {"b", 128, 1000}; }
}
static int g_calls = 0, g_failing = -1;   // the runtime's calls so far, and the one that fails
static cudaError_t next_call() { return g_calls++ == g_failing ? cudaErrorUnknown : cudaSuccess; }
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return next_call(); }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) { *n = 3; return next_call(); }
void failing(int call) { g_failing = call; g_calls = 0; }
size_t bytes(int d, int rows) { return pkv::decode_int4_workspace_bytes(64, d, rows); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("setup")
    (at / "runtime.cpp").write_text(RUNTIME)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    r = subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", cuda, "-I", build.INCLUDE, "-I", build.CSRC,
                        str(at / "runtime.cpp"), "-o", str(at / "setup.so")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    so = ctypes.CDLL(str(at / "setup.so"))
    so.bytes.restype = ctypes.c_size_t
    return so


@pytest.mark.parametrize("d,rows", [(128, 4), (128, 8), (128, 16), (64, 32), (64, 64), (64, 8)])
@pytest.mark.parametrize("call", range(6))
def test_a_failing_call_is_asked_again(lib, d, rows, call):
    fresh = _fresh(lib)
    fresh.failing(-1)
    want = fresh.bytes(d, rows)
    assert want > 0
    other = _fresh(lib)
    other.failing(call)
    assert other.bytes(d, rows) == 0
    other.failing(-1)
    assert other.bytes(d, rows) == want


def _fresh(lib):
    """Another copy of the library, with nothing set up."""
    _fresh.n = getattr(_fresh, "n", 0) + 1
    copy = f"{lib._name}.{_fresh.n}.so"
    shutil.copy(lib._name, copy)
    so = ctypes.CDLL(copy)
    so.bytes.restype = ctypes.c_size_t
    return so
