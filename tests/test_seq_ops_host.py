"""Host logic of the sequence operators that needs no GPU: refusals before any
CUDA call, and the wrapper's reading of tensor layouts."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from recurrent_cell_unroll_gb300 import _build, binding


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(_build.build())
    for name, (res, args) in binding.signatures().items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


SEQ = [n for n in binding.EXPORTED if n.startswith(("rcu_seq_", "rcu_linrec_", "rcu_layernorm_",
                                                    "rcu_act8_"))]


def test_null_handles_are_refused(lib):
    assert len(SEQ) == 14
    for name in SEQ:
        args = binding.signatures()[name][1]
        zeros = [0 if a in (ctypes.c_int, ctypes.c_int64) else 0.0 if a is ctypes.c_double else None
                 for a in args]
        rc = getattr(lib, name)(*zeros)
        if name == "rcu_seq_destroy":  # like free(NULL)
            assert rc == binding.RCU_OK
            continue
        assert rc == binding.RCU_ERR_INVALID, name
        msg = lib.rcu_last_error().decode()
        assert msg.startswith(name) and "NULL" in msg, (name, msg)


def rows(t, shape=None):
    """SeqOps._rows without a device."""
    me = SimpleNamespace(_on=lambda t, name: None)
    return binding.SeqOps._rows(me, t, "t", t.dtype, shape or t.shape)


def test_evenly_spaced_rows_are_used_in_place():
    wide = torch.arange(4 * 6 * 20, dtype=torch.float32).view(4, 6, 20)
    part = wide[..., 5:13]
    kept, ptr, ld = rows(part)
    assert kept is part and ptr == part.data_ptr() and ld == 20
    assert rows(wide)[2] == 20 and rows(wide)[0] is wide


@pytest.mark.parametrize("make", [
    lambda w: w[:, :4, :8],             # rows of unequal spacing
    lambda w: w.transpose(0, 1),        # another order
    lambda w: w[..., ::2],              # values apart
    lambda w: w[:1].expand(4, 6, 20),   # rows that overlap
    lambda w: w[:, :1, :8].expand(4, 6, 8),
    lambda w: w[0, 0, ::2],             # one row, values apart
])
def test_other_layouts_are_copied(make):
    t = make(torch.randn(4, 6, 20))
    kept, ptr, ld = rows(t)
    assert kept is not t and kept.is_contiguous() and torch.equal(kept, t) and ld == t.shape[-1]


def test_operands_are_checked_before_the_call():
    with pytest.raises(ValueError):
        rows(torch.zeros(3, 4), (3, 5))
    with pytest.raises(ValueError):  # not on a GPU
        binding.SeqOps._on(SimpleNamespace(device=0), torch.zeros(3), "x")
    with pytest.raises(ValueError):
        binding.SeqOps._tbh((3, 4), False)
    assert binding.SeqOps._tbh((3, 4, 5), False) == (3, 4, 5)
    assert binding.SeqOps._tbh((3, 4, 5), True) == (4, 3, 5)
