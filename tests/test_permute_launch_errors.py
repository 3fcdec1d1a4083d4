"""A launch of the dispatch maps that fails is the call's result and ends its chain: the
host code of permute.cu, linked to a runtime whose n-th launch returns an error."""

import ctypes
import os
import shutil
import subprocess

import pytest

FAKE = r"""
#include "moe.h"
#include <stddef.h>
struct CUstream_st;
namespace moe {
int launch_permute_maps(const moe_config_t&, const int32_t*, const float*, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*,
                        int32_t*, float*, int*, CUstream_st*, bool);
int launch_chunk_hist(const moe_config_t&, const int32_t*, int32_t*, int*, CUstream_st*);
}
static int launches, failing, last;
static int launch() {
  const int e = ++launches == failing ? 2 : 0;   // 2: cudaErrorMemoryAllocation
  if (e) last = e;                               // what cudaGetLastError returns once
  return e;
}
static void* handle;
extern "C" {
int __cudaLaunchKernel(...) { return launch(); }
int cudaLaunchKernel(...) { return launch(); }
int cudaLaunchKernelExC(...) { return launch(); }
int cudaGetLastError() { const int e = last; last = 0; return e; }
int cudaMemsetAsync(...) { return 0; }
int __cudaGetKernel(...) { return 0; }
unsigned __cudaPushCallConfiguration(...) { return 0; }
int __cudaPopCallConfiguration(...) { return 0; }
void** __cudaRegisterFatBinary(...) { return &handle; }
void __cudaRegisterFatBinaryEnd(...) {}
void __cudaUnregisterFatBinary(...) {}
void __cudaRegisterFunction(...) {}
int run(const moe_config_t* c, int fail, int hist_ready, int* count) {
  int32_t* p = reinterpret_cast<int32_t*>(1 << 20);
  float* f = reinterpret_cast<float*>(p);
  launches = last = 0;
  failing = fail;
  const int e = moe::launch_permute_maps(*c, p, f, p, p, p, p, p, p, f, p, nullptr, hist_ready != 0);
  *count = launches;
  return e;
}
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from mixture_experts_layer_softmax_gb300 import _build
    _build.build()
    d = tmp_path_factory.mktemp("fake_runtime")
    (d / "fake.cpp").write_text(FAKE)
    # (-Bsymbolic: its own functions, whatever runtime the process has loaded)
    subprocess.run([shutil.which("g++") or "g++", "-shared", "-fPIC", "-O1", "-Wl,-Bsymbolic", "-I", _build.INCLUDE,
                    str(d / "fake.cpp"), os.path.join(_build.OUT, "permute.o"), "-o", str(d / "fake.so")], check=True)
    return ctypes.CDLL(str(d / "fake.so")).run


@pytest.mark.parametrize("T,E,hist_ready,launches", [(64, 8, 0, 2), (64, 8, 1, 1), (16384, 128, 0, 3), (16384, 128, 1, 2)])
def test_each_launch(run, T, E, hist_ready, launches):
    from mixture_experts_layer_softmax_gb300 import moe as M
    cfg, count = M.make_config(T, 128, E, 2, 128), ctypes.c_int()
    assert run(ctypes.byref(cfg), 0, hist_ready, ctypes.byref(count)) == 0 and count.value == launches
    for n in range(1, launches + 1):
        assert run(ctypes.byref(cfg), n, hist_ready, ctypes.byref(count)) == 2, n
        assert count.value == n
