"""The sequence operators in the library's RCU_DEBUG build: its device bounds checks stay
silent on valid calls in every form of the recurrence (short sequences, whole rows,
clusters, shares, segments; rows that TMA can and cannot address), and its results are
those of the ordinary build's tests.  In a child process, since a process loads one
library."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import torch
sys.path[:0] = [ROOT, ROOT + "/tests"]
from recurrent_cell_unroll_gb300 import _build, binding
binding.load(_build.build(debug=True))
from test_gpu_seq_ops import check_ln, check_rec
ops = binding.SeqOps()
for force in (0, 1):
    ops.set_attr(binding.RCU_ATTR_FORCE_PATH, force)
    for dtype in ("f32", "bf16"):
        for T, B, H, lengths, act in (
                (9, 310, 66, False, False), (130, 3, 77, True, True), (300, 4, 64, True, False),
                (130, 500, 40, True, False), (4111, 2, 72, True, True), (12345, 1, 33, False, False),
                (0, 2, 8, False, False)):
            ln = [(7 * b + T) % (T + 1) for b in range(B)] if lengths else None
            check_rec(ops, T, B, H, dtype, lengths=ln, act=act)  # asserts a silent status too
        check_ln(ops, 33, 1000, dtype, True, act=True)
        check_ln(ops, 2, 9000, dtype, False)
x = torch.randn(3, 64, device="cuda")
ops.linrec_step(x, x, x, x[0], x.clone())
assert ops.status() == 0
ops.close()
print("debug build ok")
"""


def test_debug_build_checks_stay_silent():
    code = "ROOT = %r\n" % ROOT + CHILD
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "debug build ok" in r.stdout
