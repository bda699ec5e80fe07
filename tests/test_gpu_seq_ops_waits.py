"""The recurrence's bounded waits on the GPU: each gives up on what nothing brings (a copy,
a cluster's round, a carry), and is reported, over a length out of range too, after
which results would still stand."""
import ctypes
import subprocess

import pytest

from recurrent_cell_unroll_gb300 import _build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "linrec_tile.cuh"
using namespace rcu;
using namespace rcu::linrec;
// one thread; mem: a block's flag of carries, which stays 0, and its 32 carries
__global__ void wait_for(int which, void *mem, int *err, int *gave_up) {
  __shared__ uint64_t bar;
  __shared__ int abort;
  abort = 0;
  tc::mbar_init(&bar, 1);  // and nothing arrives
  tc::fence_mbar_init();
  if (which == 0) wait_copy(&bar, 0, err, &abort);
  if (which == 1) wait_round(&bar, 0, err, &abort);
  if (which == 2) take_carry<float>(mem, 0, err, &abort);
  *gave_up = abort;
}
extern "C" __attribute__((visibility("default"))) int run(int which, int before, int *after, int *gave_up) {
  int *dev = nullptr;  // err, gave_up, then (16-byte aligned) the flag and the carries
  const size_t bytes = 32 + carry_flags(1) + 32 * sizeof(float);
  cudaError_t e = cudaMalloc(&dev, bytes);
  if (e == cudaSuccess) e = cudaMemset(dev, 0, bytes);
  if (e == cudaSuccess) e = cudaMemcpy(dev, &before, 4, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) {
    wait_for<<<1, 1>>>(which, dev + 8, dev, dev + 1);
    e = cudaDeviceSynchronize();
  }
  int out[2] = {};
  if (e == cudaSuccess) e = cudaMemcpy(out, dev, 8, cudaMemcpyDeviceToHost);
  cudaFree(dev);
  *after = out[0], *gave_up = out[1];
  return (int)e;
}
"""
OK, TIMEOUT, LENGTHS = 0, 1, 2  # DevErr


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    at = tmp_path_factory.mktemp("waits")
    (at / "waits.cu").write_text(SOURCE)
    so = at / "waits.so"
    r = subprocess.run([_build.nvcc(), *_build._flags(), "-shared", "-cudart", "static", "-o", str(so),
                        str(at / "waits.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    lib = ctypes.CDLL(str(so))

    def call(which, before):
        after, gave_up = ctypes.c_int(), ctypes.c_int()
        assert lib.run(which, before, ctypes.byref(after), ctypes.byref(gave_up)) == 0
        return after.value, gave_up.value
    return call


@pytest.mark.parametrize("which", [0, 1, 2], ids=["copy", "round", "carry"])
@pytest.mark.parametrize("before,after", [(OK, TIMEOUT), (LENGTHS, TIMEOUT)])
def test_a_wait_that_ran_out_is_reported(run, which, before, after):
    assert run(which, before) == (after, 1)
