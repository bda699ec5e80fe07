"""Checks of the sequence operators' kernel sources that the CUDA compiler makes
(no GPU needed)."""
import os
import subprocess

import pytest

from recurrent_cell_unroll_gb300 import _build


def compiles(tmp_path, name, source):
    """(whether nvcc's front ends take the source, what they say)"""
    src = tmp_path / f"{name}.cu"
    src.write_text(source)
    cmd = [_build.nvcc(), _build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.INCLUDE,
           "-I", _build.CSRC, "-O0", "-ptx", "-o", os.devnull, str(src)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    return r.returncode == 0, r.stdout + r.stderr


GATES = """
#include "linrec_bwd.cuh"
using namespace rcu::linrec;
__global__ void kernel(const uint32_t *in, {v} *out) {{
  uint32_t raw[3][{n}];
  float scale[3][{n}] = {{}};
  for (int k = 0; k < 3; ++k)
    for (int s = 0; s < {n}; ++s) raw[k][s] = in[k * {n} + s];
  {v} k2, em1[{n}], nb[{n}], ns[{n}], ng[{n}];
  set(k2, 1.f);
  gates<{t}, true, {batch}>(raw, scale, k2, Limits{{}}, em1, nb, ns, ng);
  for (int s = 0; s < {n}; ++s) out[s] = em1[s];
}}
"""


@pytest.mark.parametrize("t,v,batch,n,good", [
    ("float", "float", 2, 4, True), ("bf16", "F2", 4, 4, True),
    ("float", "float", 4, 4, False),  # eight steps at once of arrays of four
    ("bf16", "F2", 4, 6, False)])
def test_gates_are_made_of_whole_batches(tmp_path, t, v, batch, n, good):
    ok, said = compiles(tmp_path, "gates", GATES.format(t=t, v=v, batch=batch, n=n))
    assert ok == good, said
    assert good or "batches" in said, said
