"""How the selective scan's kernels are told to read b and c: by words where rows are
aligned for it.  The library's own objects are linked with a stand-in for the CUDA runtime
that keeps what each scan kernel is launched with; no kernel runs, and no GPU is needed."""
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
#include "ssm.h"
namespace {
struct Segments { int n, len; };
struct Meeting { Segments seg; float *end, *sums; };
struct Forward {  // the arguments of selscan_fwd.cu's kernels
  rcu::ScanIn in;
  rcu::SeqIn dy;
  const float *h0;
  rcu::SeqOut y;
  float *h_n, *states;
  Meeting m;
  int groups;
  bool wide_states, wide_bc;
};
int count, by_words, others;
}
extern "C" {
void fake_start() { count = by_words = others = 0; }
int fake_count() { return count; }
int fake_by_words() { return by_words; }
int fake_others() { return others; }
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaMalloc(void **p, size_t n) { *p = aligned_alloc(256, (n + 255) / 256 * 256); return cudaSuccess; }
cudaError_t cudaFree(void *p) { free(p); return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return "refused"; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *, int, size_t, unsigned) {
  *n = 2;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **args) {
  if (!c->dynamicSmemBytes) return cudaSuccess;  // sums and chains
  const Forward &a = *static_cast<const Forward *>(args[0]);
  if (a.in.H == 72 && a.groups == 2) ++count, by_words += a.wide_bc;
  else ++others;
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
    src = at / "runtime.cc"
    src.write_text(RUNTIME)
    rest = at / "rest.c"  # what these calls do not need: succeeds, and does nothing
    rest.write_text("".join(f"int {n}(void) {{ return 0; }}\n" for n in sorted(wanted - mine)))
    inc = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    so = at / "librcu_fake.so"
    for cmd in (["g++", "-std=c++17", "-fPIC", "-I", inc, "-I", _build.CSRC, "-I", _build.INCLUDE, "-c", str(src),
                 "-o", str(at / "a.o")],
                ["gcc", "-fPIC", "-w", "-fno-builtin", "-c", str(rest), "-o", str(at / "b.o")],
                ["g++", "-shared", "-Wl,-Bsymbolic", "-o", str(so), str(at / "a.o"), str(at / "b.o"), *objs,
                 "-lpthread", "-ldl", "-lrt"]):
        subprocess.run(cmd, check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(str(so))
    for name, (res, args) in binding.signatures().items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


P = 1 << 20


@pytest.mark.parametrize("dtype", [binding.RCU_F32, binding.RCU_BF16])
@pytest.mark.parametrize("N,off,ld,words", [(16, 0, 16, True), (4, 0, 20, True), (16, 4, 16, False),
                                            (16, 0, 18, False), (6, 0, 8, False), (7, 0, 7, False)])
def test_forward_reads_b_and_c_by_words(lib, dtype, N, off, ld, words):
    """T=100: the main kernel; T=5000: a kernel for the segments' ends before it.  Of fp32;
    bf16 is faster value by value."""
    H = 72
    h = ctypes.c_void_p()
    assert lib.rcu_seq_create(ctypes.byref(h)) == 0
    for force in (0, 1):
        assert lib.rcu_seq_set_attr(h, binding.RCU_ATTR_FORCE_PATH, force) == 0
        for T, kernels in ((100, 1), (5000, 2)):
            lib.fake_start()
            assert lib.rcu_selscan_forward(h, dtype, 0, T, 1, H, N, P, H, P, H, P, P + off, ld, P + off, ld, None, None,
                                           None, 0, None, None, P, H, None, P, None) == 0
            assert (lib.fake_count(), lib.fake_others()) == (kernels, 0)
            assert lib.fake_by_words() == (kernels if words and not force and dtype == binding.RCU_F32 else 0)
    lib.rcu_seq_destroy(h)
