"""Tests of what is launched: on the host, with a stand-in for the CUDA runtime's
launch calls, which takes note of them and holds clusters of a given size at most;
on the GPU, with one for the question which clusters it holds."""
import json
import os
import shutil
import subprocess
import sys

import pytest

from tests.test_abi import B  # noqa: F401  (the fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_IN = r"""
#include <cuda_runtime_api.h>
#include <stdlib.h>
static int taken, sizes[64];
static int cluster(const cudaLaunchConfig_t* c) {
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return (int)c->attrs[i].val.clusterDim.x;
  return 1;
}
static int most(void) { return atoi(getenv("MOST")); }
extern "C" {
int launches(int* out) { for (int i = 0; i < taken; ++i) out[i] = sizes[i]; return taken; }
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, enum cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaPeekAtLastError(void) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  *n = cluster(c) <= most();
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**) {
  const int n = cluster(c);
  if ((n > 1 && n > most()) || c->gridDim.x % n) return cudaErrorInvalidConfiguration;
  sizes[taken++] = n;
  return cudaSuccess;
}
}
"""

NARROW = r"""
#include <cuda_runtime_api.h>
#include <stdlib.h>
extern "C" cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  int size = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) size = (int)c->attrs[i].val.clusterDim.x;
  *n = size <= atoi(getenv("MOST"));
  return cudaSuccess;
}
"""

CALLS = r"""
import ctypes, json, sys
lib, shim = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
at, big = p(1 << 20), sz(1 << 28)
def repack(freed):
    f = at if freed else None
    return lib.mla_repack_requests(at, at, i64(500), i32(3), at, i32(2), None, None, i32(0), at, at, i64(500), i64(1000), f,
                                   i64(500 if freed else 0), f, at, big, None)
def compact():
    return lib.mla_compact_cache(at, None, i64(1000), i64(1000), i32(2), i32(576), at, i32(3), at, i64(500), at, at, at,
                                 big, None)
out, before = [], 0
for call in (lambda: repack(False), lambda: repack(True), compact):
    st, got = call(), (ctypes.c_int * 64)()
    n = shim.launches(got)
    out.append((st, list(got[before:n])))
    before = n
print(json.dumps(out))
"""


def _compile(d, source):
    gxx, nvcc = shutil.which("g++"), shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if not gxx or not os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
        pytest.skip("no host compiler or CUDA headers")
    src, lib = d / "stand_in.cpp", d / "stand_in.so"
    src.write_text(source)
    subprocess.run([gxx, "-shared", "-fPIC", "-I", include, str(src), "-o", str(lib)], check=True)
    return str(lib)


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory, B):  # noqa: F811
    return _compile(tmp_path_factory.mktemp("stand_in"), STAND_IN)


def _calls(stand_in, most):
    from mla_latent_kv_absorbed_gb300 import build
    r = subprocess.run([sys.executable, "-c", CALLS, build.LIB, stand_in], capture_output=True, text=True,
                       env=dict(os.environ, LD_PRELOAD=stand_in, MOST=str(most), CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


@pytest.mark.parametrize("most", [16, 8, 2, 1])
def test_slot_scans_take_the_cluster_that_fits(stand_in, most):
    # all of a chain's kernels are launched, whatever cluster the device holds
    assert _calls(stand_in, most) == [[0, [1]], [0, [1, 1, most]], [0, [1, most, 1]]]


def test_nothing_is_marked_where_no_cluster_fits(stand_in):
    # the marks would stay in the workspace: an error, and no launch
    assert _calls(stand_in, 0)[1:] == [[4, []], [4, []]]


LIMITS = r"""
import ctypes, json, sys
lib, shim = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
at, big = p(1 << 20), sz(1 << 28)
def verify(vocab):
    return lib.mla_verify_drafts(at, i64(0), i64(0), None, i64(0), i64(0), at, None, at, i32(1), i32(1), i32(vocab), at, at, at,
                                 None, None)
def repack(new, room):
    return lib.mla_repack_requests(at, at, i64(500), i32(3), at, i32(new), None, None, i32(0), at, at, i64(room), i64(1000),
                                   None, i64(0), None, at, big, None)
top = 2**31 - 1
st = [verify(2**30), verify(2**30 + 1), verify(top), repack(2**20, 500), repack(2**20 + 1, 500), repack(top, 500),
      repack(2, top - 1), repack(2, top)]
print(json.dumps([st, shim.launches((ctypes.c_int * 64)())]))
"""


def test_sizes_that_32_bits_do_not_count_are_refused(stand_in):
    # the last block of a row, the windows of new requests and the sum of their lengths: one more would wrap around
    from mla_latent_kv_absorbed_gb300 import build
    r = subprocess.run([sys.executable, "-c", LIMITS, build.LIB, stand_in], capture_output=True, text=True,
                       env=dict(os.environ, LD_PRELOAD=stand_in, MOST="16", CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, r.stderr
    st, launched = json.loads(r.stdout)
    assert st == [0, 2, 2, 0, 2, 2, 0, 1] and launched == 3


@pytest.mark.gpu
@pytest.mark.parametrize("most", [8, 1])
def test_scans_of_smaller_clusters_give_the_same(tmp_path, most):
    lib = _compile(tmp_path, NARROW)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_between_steps.py", "-k", "repack or compact or workspace"], cwd=ROOT,
                       capture_output=True, text=True, env=dict(os.environ, LD_PRELOAD=lib, MOST=str(most)))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
