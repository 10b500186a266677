"""The host's launch helpers against a runtime whose calls are replaced at link time (CPU only)."""
import os
import subprocess

import pytest

from structured_sparse_gemm_02_b200 import build

# Replaced calls: launches and attributes fail where `fail` is set, and leave their status
# behind for the next cudaGetLastError, as the runtime does.
PRELUDE = r"""
#include <cstdio>
#include <map>
#include <utility>
#include "gather.cuh"
static bool fail = false;
static int device = 0;
static cudaError_t last = cudaSuccess;
static std::map<std::pair<int, const void*>, int> limits;
static int lowered = 0, sets = 0;
static cudaError_t status() {
  if (fail) last = cudaErrorInvalidValue;
  return fail ? cudaErrorInvalidValue : cudaSuccess;
}
extern "C" {
cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return status(); }
cudaError_t __wrap_cudaGetDevice(int* dev) { *dev = device; return status(); }
cudaError_t __wrap_cudaFuncSetAttribute(const void* k, cudaFuncAttribute, int v) {
  int& now = limits[{device, k}];
  ++sets;
  lowered += v < now;
  now = v;
  return status();
}
cudaError_t __wrap_cudaGetLastError() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
}
__global__ void kernel(int) {}
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    def f(body):
        d = tmp_path_factory.mktemp("prog")
        src, exe = d / "prog.cu", d / "prog"
        src.write_text(PRELUDE + "int main() {\n" + body + "\nreturn 0;\n}\n")
        wraps = [w for name in ("cudaLaunchKernelExC", "cudaGetDevice", "cudaFuncSetAttribute", "cudaGetLastError")
                 for w in ("-Xlinker", f"--wrap={name}")]
        subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, str(src),
                        os.path.join(build.CSRC, "api.cu"), *wraps, "-o", str(exe), "-ldl", "-lpthread", "-lrt"],
                       check=True, capture_output=True, text=True)
        p = subprocess.run([str(exe)], capture_output=True, text=True)
        assert p.returncode == 0, p.stdout + p.stderr
    return f


def test_a_failed_call_leaves_no_status_for_the_next_one(run):
    run(r"""
  fail = true;
  CHECK(spg::launch_pdl(kernel, dim3(1), dim3(32), 0, nullptr, 1) == cudaErrorInvalidValue);
  CHECK(spg::launch_status() == SPG_OK);
  CHECK(spg::launch_pdl_cluster(kernel, dim3(2), dim3(32), 0, 2, nullptr, 1) == cudaErrorInvalidValue);
  CHECK(spg::launch_status() == SPG_OK);
  CHECK(spg::allow_smem(reinterpret_cast<const void*>(kernel), 65536) != cudaSuccess);
  CHECK(spg::launch_status() == SPG_OK);
  fail = false;
  CHECK(spg::launch_pdl(kernel, dim3(1), dim3(32), 0, nullptr, 1) == cudaSuccess);
  CHECK(spg::allow_smem(reinterpret_cast<const void*>(kernel), 65536) == cudaSuccess);
""")


def test_shared_memory_limits_of_many_kernels_and_devices_never_fall(run):
    """A limit is set once for each kernel and device, raised for a larger launch and never lowered."""
    run(r"""
  static char kernels[200];
  for (device = 0; device < 8; ++device)
    for (char& k : kernels) CHECK(spg::allow_smem(&k, 100000) == cudaSuccess);
  CHECK(sets == 8 * 200);
  for (device = 0; device < 8; ++device)
    for (char& k : kernels) {
      CHECK(spg::allow_smem(&k, 60000) == cudaSuccess);
      CHECK(spg::allow_smem(&k, 100000) == cudaSuccess);
    }
  CHECK(lowered == 0 && sets == 8 * 200);
  device = 3;
  CHECK(spg::allow_smem(kernels + 150, 120000) == cudaSuccess && sets == 8 * 200 + 1);
""")
