"""Host logic of the sequence operators that needs no GPU: refusals before any
CUDA call, and the wrapper's reading of tensor layouts."""
import ctypes

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
    """SeqOps._rows of a tensor taken to be on the handle's device (that of a
    host tensor is -1): (pointer, row stride, the copy if one was made)."""
    me = object.__new__(binding.SeqOps)
    me.h, me.device = None, -1
    me._refuse_or_copy = lambda t, name, dtype, shape, keep: \
        keep.append(t.clone(memory_format=torch.contiguous_format)) or keep[0]
    keep = []
    return (*me._rows(t, "t", t.dtype, shape or t.shape, keep), keep[0] if keep else None)


def test_evenly_spaced_rows_are_used_in_place():
    wide = torch.arange(4 * 6 * 20, dtype=torch.float32).view(4, 6, 20)
    part = wide[..., 5:13]
    assert rows(part) == (part.data_ptr(), 20, None)
    assert rows(wide) == (wide.data_ptr(), 20, None)


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
    ptr, ld, copy = rows(t)
    assert copy.is_contiguous() and torch.equal(copy, t)
    assert ptr == copy.data_ptr() and ld == t.shape[-1]


def test_operands_are_checked_before_the_call():
    me = object.__new__(binding.SeqOps)
    me.h, me.device = None, 0
    x = torch.zeros(3, 4)
    for call in (lambda: me._rows(x, "x", x.dtype, x.shape, []),        # not on a GPU
                 lambda: me._dense(x, "x", x.dtype, x.shape, []),
                 lambda: me._dense([1.0], "x", x.dtype, x.shape, []),
                 lambda: me._type(None, "x"), lambda: me._type(x.half(), "x"),
                 lambda: me._type(x, "x", 3), lambda: me._type(torch.zeros(()), "x")):
        with pytest.raises(ValueError):
            call()
    assert me._type(x, "x", 2) == (torch.float32, binding.RCU_F32, x.shape)
