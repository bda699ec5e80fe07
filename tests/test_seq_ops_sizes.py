"""Sizes that the sequence operators' kernels cannot count are refused before a launch
(against a stand-in for the CUDA runtime: no GPU needed)."""
import ctypes

import pytest

from recurrent_cell_unroll_gb300 import binding
from test_seq_ops_devices import P, lib  # noqa: F401 (fixture)

UNSUPPORTED = binding.RCU_ERR_UNSUPPORTED


@pytest.fixture
def handle(lib):  # noqa: F811
    lib.fake_device(0)
    h = ctypes.c_void_p()
    assert lib.rcu_seq_create(ctypes.byref(h)) == binding.RCU_OK
    yield h
    lib.rcu_seq_destroy(h)


# A row's columns are counted in 32 bits, and rounded up to tiles and blocks.
@pytest.mark.parametrize("n,code", [((1 << 31) - 8192, 0), ((1 << 31) - 8191, UNSUPPORTED), ((1 << 31) - 40, UNSUPPORTED),
                                    ((1 << 31) - 1, UNSUPPORTED)])
def test_widths(lib, handle, n, code):  # noqa: F811
    h = handle
    assert lib.rcu_linrec_forward(h, 0, 0, 1, 1, n, P, n, P, n, P, n, P, 8.0, None, None, P, n, None, None,
                                  None) == code
    assert lib.rcu_linrec_backward(h, 0, 0, 0, 1, 1, n, P, n, P, n, P, n, None, None, None, P, 8.0, None, P, P, n,
                                   None, P, n, P, n, P, n, None, None, None) == code
    assert lib.rcu_linrec_step(h, 0, 1, n, P, n, P, n, P, n, P, 8.0, P, 1, None, P, n, None) == code
    assert lib.rcu_layernorm_forward(h, 0, 1, n, P, n, None, 0, None, None, 1e-5, P, n, None, 0, None, None,
                                     None) == code
    assert lib.rcu_layernorm_backward(h, 0, 0, 1, n, P, n, P, n, None, None, P, P, None, 0, P, n, None, None,
                                      None) == code
    assert lib.rcu_act8_pack(h, 0, 1, n, P, n, P, n, P, None) == code
    assert lib.rcu_act8_unpack(h, 0, 1, n, P, n, P, P, n, None) == code
