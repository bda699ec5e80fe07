"""Host logic of the selective state space operators and of the AdamW step that needs no
GPU: refusals before any CUDA call, sizes beyond what the kernels count, and the kernels'
limits on a process with two devices (against a stand-in for the CUDA runtime)."""
import ctypes

import pytest
import torch

from recurrent_cell_unroll_gb300 import binding
from test_seq_ops_devices import P, lib  # noqa: F401 (fixture)

INVALID, UNSUPPORTED = binding.RCU_ERR_INVALID, binding.RCU_ERR_UNSUPPORTED
NEW = [n for n in binding.EXPORTED if n.startswith(("rcu_conv_", "rcu_selscan_", "rcu_adamw_", "rcu_state8_"))]


@pytest.fixture
def handle(lib):  # noqa: F811
    lib.fake_device(0)
    h = ctypes.c_void_p()
    assert lib.rcu_seq_create(ctypes.byref(h)) == 0
    yield h
    lib.fake_device(0)
    lib.rcu_seq_destroy(h)


def conv_fwd(lib, h, T, B, H, W, dtype=0, layout=0, ld=None, x=P, w=P, y=P):  # noqa: F811
    ld = H if ld is None else ld
    return lib.rcu_conv_forward(h, dtype, layout, T, B, H, W, x, ld, w, None, 1, None, None, y, H, P, None)


def conv_bwd(lib, h, T, B, H, W, dtype=0, ds=P, dsn=None):  # noqa: F811
    return lib.rcu_conv_backward(h, dtype, 0, T, B, H, W, P, H, P, None, 1, None, None, P, H, dsn, P, H, P, P, ds,
                                 None)


def scan_fwd(lib, h, T, B, H, N, dtype=0, p=P, x=P, a=P, ldb=None):  # noqa: F811
    return lib.rcu_selscan_forward(h, dtype, 0, T, B, H, N, x, H, p, H, a, p, N if ldb is None else ldb, p, N, P, P, p,
                                   H, None, None, p, H, P, P, None)


def scan_bwd(lib, h, T, B, H, N, dtype=0, p=P, states=P, z=P, d=P):  # noqa: F811
    return lib.rcu_selscan_backward(h, dtype, 0, T, B, H, N, p, H, p, H, P, p, N, p, N, d, P, z, H, None, states, p, H,
                                    None, p, H, p, H, P, p, N, p, N, P, P, P, H, P, None)


def test_null_handles_are_refused(lib):  # noqa: F811
    assert len(NEW) == 9
    for name in NEW:
        args = binding.signatures()[name][1]
        zeros = [0 if a in (ctypes.c_int, ctypes.c_int64) else 0.0 if a is ctypes.c_double else None for a in args]
        assert getattr(lib, name)(*zeros) == INVALID
        msg = lib.rcu_last_error().decode()
        assert msg.startswith(name) and "NULL" in msg, msg


def test_sizes(lib, handle):  # noqa: F811
    h = handle
    for T, B, H, code in ((1, 1, 8, 0), (0, 3, 8, 0), (3, 0, 8, 0), (-1, 1, 8, INVALID), (1, -1, 8, INVALID),
                          (1, 1, 0, INVALID), ((1 << 30) + 1, 1, 8, UNSUPPORTED), (1 << 20, 1 << 10, 1, UNSUPPORTED),
                          (1, 1 << 20, 1 << 10, UNSUPPORTED)):
        assert conv_fwd(lib, h, T, B, H, 4) == code and conv_bwd(lib, h, T, B, H, 4) == code, (T, B, H)
        assert scan_fwd(lib, h, T, B, H, 16) == code and scan_bwd(lib, h, T, B, H, 16) == code, (T, B, H)
    for n, code in ((0, INVALID), (9, UNSUPPORTED), (8, 0), (1, 0)):
        assert conv_fwd(lib, h, 4, 2, 8, n) == code and conv_bwd(lib, h, 4, 2, 8, n) == code
        assert lib.rcu_conv_step(h, 0, 2, 8, n, P, 8, P, None, 1, P, 2, None, P, 8, None) == code
    for n, code in ((0, INVALID), (65, UNSUPPORTED), (64, 0), (1, 0)):
        assert scan_fwd(lib, h, 4, 2, 8, n) == code and scan_bwd(lib, h, 4, 2, 8, n) == code
        assert lib.rcu_selscan_step(h, 0, 2, 8, n, P, 8, P, 8, P, P, 64, P, 64, None, None, None, 0, P, 2, None, P, 8,
                                    None) == code


def test_missing_and_overlapping_operands(lib, handle):  # noqa: F811
    h = handle
    assert conv_fwd(lib, h, 4, 2, 8, 4, dtype=2) == INVALID
    assert conv_fwd(lib, h, 4, 2, 8, 4, layout=2) == INVALID
    assert conv_fwd(lib, h, 4, 2, 8, 4, ld=7) == INVALID
    assert conv_fwd(lib, h, 4, 2, 8, 4, x=None) == INVALID
    assert conv_fwd(lib, h, 4, 2, 8, 4, w=None) == INVALID
    assert conv_fwd(lib, h, 4, 2, 8, 4, y=None) == INVALID
    assert conv_bwd(lib, h, 4, 2, 8, 4, ds=P, dsn=P) == INVALID
    assert scan_fwd(lib, h, 4, 2, 8, 4, x=None) == INVALID
    assert scan_fwd(lib, h, 4, 2, 8, 4, a=None) == INVALID
    assert scan_fwd(lib, h, 4, 2, 8, 4, ldb=3) == INVALID
    assert scan_bwd(lib, h, 4, 2, 8, 4, states=None) == INVALID
    assert scan_bwd(lib, h, 4, 2, 8, 4, z=None) == INVALID   # dz is asked for
    assert scan_bwd(lib, h, 4, 2, 8, 4, d=None) == INVALID   # dd is
    # fewer state rows than requests without slots
    assert lib.rcu_conv_step(h, 0, 3, 8, 4, P, 8, P, None, 1, P, 2, None, P, 8, None) == INVALID
    assert lib.rcu_conv_step(h, 0, 3, 8, 4, P, 8, P, None, 1, None, 3, None, P, 8, None) == INVALID
    assert lib.rcu_selscan_step(h, 0, 3, 8, 4, P, 8, P, 8, P, P, 4, P, 4, None, None, None, 0, P, 2, None, P, 8,
                                None) == INVALID


def test_kernels_are_set_up_on_each_device(lib):  # noqa: F811
    handles = []
    for device in (0, 1, 0, 1):
        lib.fake_device(device)
        h = ctypes.c_void_p()
        assert lib.rcu_seq_create(ctypes.byref(h)) == 0
        handles.append((device, h))
    for device, h in handles:
        lib.fake_device(device)
        for dtype in (0, 1):
            for p in (P, P + 4):  # rows that words can and cannot address
                for N in (3, 8, 16, 32, 64):
                    for T, B, H in ((100, 3, 64), (5000, 1, 128), (300, 40, 520)):
                        said = (device, dtype, p, N, T, lib.rcu_last_error())
                        assert scan_fwd(lib, h, T, B, H, N, dtype, p) == 0, said
                        assert scan_bwd(lib, h, T, B, H, N, dtype, p) == 0, said
            for W in (1, 2, 3, 4, 8):
                assert conv_fwd(lib, h, 100, 3, 64, W, dtype) == 0 and conv_bwd(lib, h, 100, 3, 64, W, dtype) == 0
        other = ctypes.c_void_p(h.value)
        lib.fake_device(1 - device)
        assert conv_fwd(lib, other, 4, 2, 8, 4) == INVALID  # another device's handle
    for device, h in handles:
        lib.fake_device(device)
        lib.rcu_seq_destroy(h)


def rows_of(*tensors):
    return (ctypes.c_int64 * (9 * len(tensors)))(*[v for t in tensors for v in t])


def step(lib, h, table, count=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, t=1, t_dev=None):  # noqa: F811
    return lib.rcu_adamw_step(h, count, table, lr, b1, b2, eps, wd, t, 0, None, t_dev, None, None)


def test_adamw_lists(lib, handle):  # noqa: F811
    h, bf16 = handle, 1 | 1 << 32
    good = (P, P, P, P, 0, 0, 0, 100, 0)
    assert step(lib, h, rows_of(good)) == 0 and lib.rcu_seq_last_launch_count(h) == 1
    assert step(lib, h, rows_of(*[good] * 1000), 1000) == 0 and lib.rcu_seq_last_launch_count(h) == 3
    assert step(lib, h, None, 0) == 0 and lib.rcu_seq_last_launch_count(h) == 0
    assert step(lib, h, rows_of((0, 0, 0, 0, 0, 0, 0, 0, 0))) == 0 and lib.rcu_seq_last_launch_count(h) == 0
    # pieces of all tensors together beyond what one launch counts
    big = (P, P, P, P, 0, 0, 0, 1 << 40, 0)
    assert step(lib, h, rows_of(*[big] * 40), 40) == 0 and lib.rcu_seq_last_launch_count(h) >= 2
    for bad, code in (((0, P, P, P, 0, 0, 0, 1, 0), INVALID), ((P, P, P, P, 0, 0, 0, -1, 0), INVALID),
                      ((P, P, P, P, P, 0, 0, 1, 0), INVALID), ((P, P, P, P, 0, 0, P, 1, bf16), INVALID),
                      ((P, P, P, P, 0, 0, 0, 1, 2), INVALID), ((P, P, P, P, P, P, 0, (1 << 32) + 1, 0), UNSUPPORTED),
                      ((P, P, P, P, 0, 0, 0, (1 << 40) + 1, 0), UNSUPPORTED)):
        assert step(lib, h, rows_of(good, bad), 2) == code, bad
    t = rows_of(good)
    assert step(lib, h, None, 1) == INVALID and step(lib, h, t, -1) == INVALID
    assert step(lib, h, t, (1 << 24) + 1) == UNSUPPORTED
    for kw in ({"b1": 1.0}, {"b2": -0.1}, {"b1": float("nan")}, {"eps": -1.0}, {"lr": float("inf")},
               {"wd": float("nan")}, {"t": 0}):
        assert step(lib, h, t, **kw) == INVALID, kw
    assert step(lib, h, t, t=0, t_dev=P) == 0


def test_state8_arguments(lib, handle):  # noqa: F811
    for fn in (lib.rcu_state8_pack, lib.rcu_state8_unpack):
        assert fn(handle, 1, 0, None, None, None, None) == 0
        assert fn(handle, 1, 100, P, P, P, None) == 0
        assert fn(handle, 1, -1, P, P, P, None) == INVALID
        assert fn(handle, 1, 1, P, None, P, None) == INVALID
        assert fn(handle, 1, (1 << 40) + 1, P, P, P, None) == UNSUPPORTED


def test_wrappers_refuse_before_the_call():
    me = object.__new__(binding.SeqOps)
    me.h, me.device = None, 0
    x, w = torch.zeros(3, 2, 4), torch.zeros(4, 3)
    for call in (lambda: me.conv_forward(x, w), lambda: me.conv_forward(x, torch.zeros(4)),
                 lambda: me.conv_forward(x[0], w), lambda: me.conv_step(x[0], w, None),
                 lambda: me.conv_step(x[0], w, torch.zeros(2, 2, 8)[..., ::2]),
                 lambda: me.selscan_forward(x, x, torch.zeros(4), x, x), lambda: me.selscan_forward(x, x, w, x, x),
                 lambda: me.selscan_step(x[0], x[0], w, x[0], x[0], None),
                 lambda: me.selscan_backward(x, x, x, w, x, x, None),
                 lambda: me.adamw_step([x], [x], [x], [x], 1), lambda: me.adamw_step([x], [], [x], [x], 1),
                 lambda: me.adamw_step([1], [x], [x], [x], 1), lambda: me.state8_pack(None, True),
                 lambda: me.state8_unpack(x, x, True)):
        with pytest.raises(ValueError):
            call()
