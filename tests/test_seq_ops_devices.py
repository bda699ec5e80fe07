"""The sequence operators' host side on a process with two devices, against a stand-in
for the CUDA runtime that keeps what belongs to a device per device: a kernel's
limits (its dynamic shared memory, its cluster size) and how much of it fits.  The
library's own objects are linked with it; no kernel runs, and no GPU is needed."""
import ctypes
import glob
import os
import re
import subprocess

import pytest

from recurrent_cell_unroll_gb300 import _build, binding

RUNTIME = r"""
#include <cuda_runtime.h>
#include <cstdlib>
#include <map>
#include <utility>
static int dev = 0;
static std::map<std::pair<int, const void *>, int> shared, wide;  // limits that were set
static std::map<int, int> grids;                                  // largest grid launched on a device
static int per_sm(int d) { return d == 0 ? 2 : 1; }               // device 1 has room for half as many
extern "C" {
void fake_device(int d) { dev = d; }
int fake_largest_grid(int d) { return grids[d]; }
cudaError_t cudaGetDevice(int *d) { *d = dev; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaMalloc(void **p, size_t n) { *p = aligned_alloc(256, (n + 255) / 256 * 256); return cudaSuccess; }
cudaError_t cudaFree(void *p) { free(p); return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return "refused"; }
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute a, int v) {
  (a == cudaFuncAttributeMaxDynamicSharedMemorySize ? shared : wide)[{dev, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *, int, size_t, unsigned) {
  *n = per_sm(dev);
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *c) {
  *n = 152 * per_sm(dev) / c->attrs[0].val.clusterDim.x;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
  const int most = shared.count({dev, f}) ? shared[{dev, f}] : 48 << 10;
  int cluster = 1, waits = 0;
  for (unsigned k = 0; k < c->numAttrs; ++k) {
    if (c->attrs[k].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[k].val.clusterDim.x;
    if (c->attrs[k].id == cudaLaunchAttributeCooperative) waits = c->attrs[k].val.cooperative;
  }
  if ((int)c->dynamicSmemBytes > most) return cudaErrorInvalidValue;
  if (cluster > 8 && !wide.count({dev, f})) return cudaErrorInvalidClusterSize;
  if (waits && (int)c->gridDim.x > 152 * per_sm(dev)) return cudaErrorCooperativeLaunchTooLarge;
  if ((int)c->gridDim.x > grids[dev]) grids[dev] = c->gridDim.x;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(void *, dim3 grid, dim3, void **, size_t smem, void *) {
  if (smem > 48 << 10) return cudaErrorInvalidValue;
  if ((int)grid.x > grids[dev]) grids[dev] = grid.x;
  return cudaSuccess;
}
static dim3 grid_of;
static size_t smem_of;
unsigned __cudaPushCallConfiguration(dim3 g, dim3, size_t s, void *) { grid_of = g; smem_of = s; return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *g, dim3 *, size_t *s, void *) { *g = grid_of; *s = smem_of; return cudaSuccess; }
static int encode() { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *r) {
  *f = (void *)encode;
  if (r) *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    _build.build()
    at = tmp_path_factory.mktemp("fake")
    objs = [os.path.join(_build.OBJDIR, os.path.basename(c)[:-3] + ".o")
            for c in sorted(glob.glob(os.path.join(_build.CSRC, "*.cu")))]
    wanted = set(re.findall(r"\bU (_*cuda\w+)", subprocess.run(["nm", "-u", *objs], capture_output=True,
                                                              text=True, check=True).stdout))
    mine = set(re.findall(r"\b(_*cuda\w+)\(", RUNTIME))
    src = at / "runtime.cu"
    src.write_text(RUNTIME)
    rest = at / "rest.c"  # what these calls do not need: succeeds, and does nothing
    rest.write_text("".join(f"int {n}(void) {{ return 0; }}\n" for n in sorted(wanted - mine)))
    inc = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    so = at / "librcu_fake.so"
    for cmd in (["g++", "-std=c++17", "-fPIC", "-I", inc, "-x", "c++", "-c", str(src), "-o", str(at / "a.o")],
                ["gcc", "-fPIC", "-w", "-fno-builtin", "-c", str(rest), "-o", str(at / "b.o")],
                ["g++", "-shared", "-Wl,-Bsymbolic", "-o", str(so), str(at / "a.o"), str(at / "b.o"), *objs,
                 "-lpthread", "-ldl", "-lrt"]):
        subprocess.run(cmd, check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(str(so))
    for name, (res, args) in binding.signatures().items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


P = 1 << 20  # stands for any tensor, aligned to 16 bytes


def forward(lib, h, dtype, T, B, H, p):
    return lib.rcu_linrec_forward(h, dtype, 0, T, B, H, p, H, p, H, p, H, P, 8.0, None, None, p, H, P, P, None)


def backward(lib, h, dtype, saved, T, B, H, p):
    e = P if saved == binding.RCU_I8 else None
    return lib.rcu_linrec_backward(h, dtype, saved, 0, T, B, H, p, H, p, H, p, H, e, e, e, P, 8.0, None, P, p, H,
                                   None, p, H, p, H, p, H, P, P, None)


SHAPES = [(1000, 500, 128), (4096, 3, 192), (65536, 1, 2048), (20000, 1, 64), (64, 600, 64), (16, 600, 128)]


def test_kernels_are_set_up_on_each_device(lib):
    handles = []
    for device in (0, 1, 0, 1):
        lib.fake_device(device)
        h = ctypes.c_void_p()
        assert lib.rcu_seq_create(ctypes.byref(h)) == binding.RCU_OK
        handles.append((device, h))
    for device, h in handles:
        lib.fake_device(device)
        for T, B, H in SHAPES:
            for p in (P, P + 4):  # rows that TMA can and cannot address
                for dtype in (binding.RCU_F32, binding.RCU_BF16):
                    said = (device, T, B, H, p, dtype)
                    assert forward(lib, h, dtype, T, B, H, p) == 0, (said, lib.rcu_last_error())
                    for saved in (dtype, binding.RCU_I8):
                        assert backward(lib, h, dtype, saved, T, B, H, p) == 0, (said, lib.rcu_last_error())
    for device, h in handles:
        lib.fake_device(device)
        lib.rcu_seq_destroy(h)


def test_layer_norm_grid_of_a_device_with_less_room(lib):
    lib.fake_device(0)
    h0, h1 = ctypes.c_void_p(), ctypes.c_void_p()
    assert lib.rcu_seq_create(ctypes.byref(h0)) == binding.RCU_OK
    lib.fake_device(2)  # has room for one block an SM, and no launch yet
    assert lib.rcu_seq_create(ctypes.byref(h1)) == binding.RCU_OK

    def norm(h):
        return lib.rcu_layernorm_forward(h, 0, 1 << 20, 128, P, 128, None, 0, None, None, 1e-5, P, 128, None, 0,
                                         None, None, None)
    lib.fake_device(0)
    assert norm(h0) == 0
    lib.fake_device(2)
    assert norm(h1) == 0
    assert lib.fake_largest_grid(2) == 152
    lib.rcu_seq_destroy(h1)
    lib.fake_device(0)
    lib.rcu_seq_destroy(h0)
