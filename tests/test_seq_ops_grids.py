"""Grids of the recurrence's kernels for short sequences (against a stand-in for the CUDA
runtime: no GPU needed)."""
import ctypes

import pytest

from recurrent_cell_unroll_gb300 import binding
from test_seq_ops_devices import P, backward, forward, lib  # noqa: F401 (fixture)


@pytest.mark.parametrize("groups", [3, 16, 17, 30, 31, 32, 33, 37, 61, 64])
def test_short_sequences_take_one_wave(lib, groups):  # noqa: F811
    """No more blocks than the stand-in's 152 SMs hold, one on each, whatever the number of
    channel groups."""
    for call, device in ((forward, 1000 + groups), (backward, 2000 + groups)):
        lib.fake_device(device)
        h = ctypes.c_void_p()
        assert lib.rcu_seq_create(ctypes.byref(h)) == binding.RCU_OK
        for B in (250, 1000):
            saved = [binding.RCU_BF16] if call is backward else []
            assert call(lib, h, binding.RCU_BF16, *saved, 4, B, 64 * groups, P) == 0
        assert 0 < lib.fake_largest_grid(device) <= 152
        lib.rcu_seq_destroy(h)
