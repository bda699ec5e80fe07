"""The selective scan where a sequence is split over time and where it is not (by itself, and
as a row of a large batch), and the short convolution's and the scan's addresses beyond 32
bits.  Tolerances as in test_gpu_ssm.py."""
import pytest
import torch

import ssm_ref as ref
from recurrent_cell_unroll_gb300 import binding
from test_gpu_ssm import Make, close, scan_inputs

pytestmark = pytest.mark.gpu

NAMES = ("dx", "ddt", "da_log", "db", "dc", "dd", "ddt_bias", "dz", "dh0")


@pytest.fixture(scope="module")
def ops():
    o = binding.SeqOps()
    yield o
    o.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 4, 5, 8, 12, 16, 32, 64])
def test_a_row_alone_and_in_a_batch(ops, dtype, N):
    """T=600 of 64 channels: alone in eight segments or more, as one of 320 rows in none."""
    T, B, H, row = 600, 320, 64, 201
    make = Make(N, dtype)
    args, leaves = scan_inputs(make, T, 1, H, N)
    dy, rdy = make(T, 1, H)
    dh, rdh = make(1, H, N, f32=True)
    want = ref.scan(*leaves[:8], None, leaves[8])[:2]
    there = [t for t in leaves if t is not None]
    grads = dict(zip(NAMES, torch.autograd.grad(want, there, (rdy, rdh), retain_graph=True)))
    apart = leaves[1].detach().requires_grad_()
    parts = ref.scan(*leaves[:8], None, leaves[8], dt_in=apart)[:2]
    terms = float(sum(t.abs() for t in torch.autograd.grad(parts, (leaves[1], apart), (rdy, rdh))).max())

    def among(t, dim):  # the row among others, at random
        if t is None:
            return None
        shape = list(t.shape)
        shape[dim] = B
        room = torch.randn(shape, generator=make.g).to(t.dtype).cuda()
        room.select(dim, row).copy_(t.select(dim, 0))
        return room
    alone = (*args, dy, dh)
    wide = [among(t, d) if d is not None else t for t, d in zip(alone, (1, 1, None, 1, 1, None, None, 1, 0, 1, 0))]
    wide[1] = wide[1].clamp(max=2.0)  # (the other rows' steps)
    wide[1][:, row] = args[1][:, 0]
    for (x, dt, al, b, c, d, db, z, h, g, gh), at in ((alone, 0), (wide, row)):
        y, h_n, states = ops.selscan_forward(x, dt, al, b, c, d=d, dt_bias=db, z=z, h0=h, states=True)
        assert ops.launch_count() == (3 if at == 0 else 1)
        close(y[:, at:at + 1], want[0], "y")
        close(h_n[at:at + 1], want[1], "h_n")
        got = ops.selscan_backward(g, x, dt, al, b, c, states, d=d, dt_bias=db, z=z, dh_n=gh)
        for name in ("dx", "ddt", "db", "dc", "dz"):
            close(got[name][:, at:at + 1], grads[name], name, terms if name == "ddt" else None)
        close(got["dh0"][at:at + 1], grads["dh0"], "dh0")
    assert ops.status() == 0


def apart(room, rows, H, far):
    return room.as_strided((rows, 1, H), (far, far, 1))


@pytest.mark.parametrize("W", [4, 6])
def test_convolution_of_rows_beyond_32_bits(ops, W):
    """Evenly spaced rows, 2^30 elements apart, in place: inputs by the binding, outputs by the C
    call."""
    H, T, far = 64, 5, 1 << 30
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    g = torch.Generator(device="cuda").manual_seed(W)
    v, dy = (torch.randn(T, 1, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(H, W, generator=g, device="cuda")
    room = torch.empty((T - 1) * far + H, dtype=torch.bfloat16, device="cuda")
    out = torch.empty((T - 1) * far + H, dtype=torch.bfloat16, device="cuda")
    x, y = apart(room, T, H, far), apart(out, T, H, far)
    assert ops._rows(x, "x", x.dtype, x.shape, []) == (room.data_ptr(), far)
    x.copy_(v)
    want, end = ops.conv_forward(v, w)
    got, end2 = ops.conv_forward(x, w)
    assert torch.equal(want, got) and torch.equal(end, end2)
    want_b = ops.conv_backward(dy, v, w)
    for p, q in zip(want_b, ops.conv_backward(dy, x, w)):
        assert torch.equal(p, q)
    s = torch.cuda.current_stream().cuda_stream
    y.fill_(float("nan"))
    assert ops.lib.rcu_conv_forward(ops.h, binding.RCU_BF16, 0, T, 1, H, W, x.data_ptr(), far, w.data_ptr(), None, 1,
                                    None, None, y.data_ptr(), far, None, s) == 0
    assert torch.equal(y, want)
    y.fill_(float("nan"))
    # dy lies far apart too: x's rows, used up by now
    x.copy_(dy)
    assert ops.lib.rcu_conv_backward(ops.h, binding.RCU_BF16, 0, T, 1, H, W, v.data_ptr(), H, w.data_ptr(), None, 1,
                                     None, None, x.data_ptr(), far, None, y.data_ptr(), far, None, None, None, s) == 0
    assert torch.equal(y, want_b[0])
    assert ops.status() == 0


def test_scan_outputs_beyond_32_bits(ops):
    """y, and each gradient of a row, 2^30 elements apart, by the C call."""
    H, N, T, far = 64, 8, 5, 1 << 30
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dt, z, dy = (torch.randn(T, 1, H, generator=g, device="cuda").bfloat16() for _ in range(4))
    b, c = (torch.randn(T, 1, N, generator=g, device="cuda").bfloat16() for _ in range(2))
    al = torch.randn(H, N, generator=g, device="cuda")
    want, _, states = ops.selscan_forward(x, dt, al, b, c, z=z, states=True)
    grads = ops.selscan_backward(dy, x, dt, al, b, c, states, z=z)
    out = torch.empty((T - 1) * far + 1024, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    y = apart(out, T, H, far)
    y.fill_(float("nan"))
    put = lambda t, n: (t.data_ptr(), n)  # noqa: E731
    ins = (*put(x, H), *put(dt, H), al.data_ptr(), *put(b, N), *put(c, N), None, None, *put(z, H), None)
    assert ops.lib.rcu_selscan_forward(ops.h, binding.RCU_BF16, 0, T, 1, H, N, *ins, None, y.data_ptr(), far, None,
                                       None, s) == 0
    assert torch.equal(y, want)
    rows = {}
    for k, (name, n) in enumerate((("dx", H), ("ddt", H), ("db", N), ("dc", N), ("dz", H))):
        rows[name] = apart(out[k * 128:], T, n, far)
        rows[name].fill_(float("nan"))
    at = {k: (t.data_ptr(), far) for k, t in rows.items()}
    assert ops.lib.rcu_selscan_backward(ops.h, binding.RCU_BF16, 0, T, 1, H, N, *ins, states.data_ptr(),
                                        *put(dy, H), None, *at["dx"], *at["ddt"], None, *at["db"], *at["dc"], None,
                                        None, *at["dz"], None, s) == 0
    for name, t in rows.items():
        assert torch.equal(t, grads[name]), name
    assert ops.status() == 0
