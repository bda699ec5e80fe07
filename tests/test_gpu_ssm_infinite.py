"""Infinite values in the selective scan: where the formulas, in 64 bits, give an infinity
or a finite number, the kernels do too, and NaN only where the formulas have it.

What a thread holds beside a call's own steps, states and channels (steps up to a multiple
of four, states up to one of four or of its kind of kernel, channels up to a block's) must
stay out of the sums over them, since 0 times an infinity is NaN.

Inputs are positive, so that no infinity meets its opposite but in the gradient of dt (the
part through the decays is negative).  Finite values: as in test_gpu_ssm.py, the gradient
of dt and its sums with their terms' magnitudes.
"""
import pytest
import torch

import ssm_ref as ref
from recurrent_cell_unroll_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16_HALF = 2e-5, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")
NAMES = ("dx", "ddt", "da_log", "db", "dc", "dd", "ddt_bias", "dz", "dh0")


@pytest.fixture(scope="module")
def ops():
    o = binding.SeqOps()
    yield o
    o.close()


@pytest.fixture(params=[0, 1], ids=["auto", "plain-loads"])
def path(ops, request):
    ops.set_attr(binding.RCU_ATTR_FORCE_PATH, request.param)
    yield request.param
    ops.set_attr(binding.RCU_ATTR_FORCE_PATH, 0)


def inputs(T, B, H, N, dtype, put, slow=-1.0):
    """(x, dt, a_log, b, c, d, dt_bias, z, h0, dy, dh_n) in 64 bits as the GPU gets them, all
    positive but dt, with the infinities of `put`: name, place.  slow: dt's mean."""
    g = torch.Generator().manual_seed(T + 100 * H + N)

    def one(shape, dtype, add=0.1):
        return (torch.rand(shape, generator=g) + add).to(dtype).double()
    t, f32 = DT[dtype], torch.float32
    v = {"x": one((T, B, H), t), "dt": one((T, B, H), t, slow), "a_log": one((H, N), f32, 0.0),
         "b": one((T, B, N), t), "c": one((T, B, N), t), "d": one((H,), f32), "dt_bias": one((H,), f32, -0.5),
         "z": one((T, B, H), t), "h0": one((B, H, N), f32), "dy": one((T, B, H), t), "dh_n": one((B, H, N), f32)}
    for name, at in put:
        v[name][at] = INF
    return v


def same(got, want, name, top=0.0):
    """Infinities and NaN in the same places, finite values close."""
    half = BF16_HALF if got.dtype == torch.bfloat16 else 0.0
    got, want = got.detach().cpu().double(), want.detach()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), \
        f"{name}: {int(torch.isnan(got).sum())} NaN, {int(torch.isnan(want).sum())} by the formula"
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{name}: infinities"
    got, want = got[fine], want[fine]
    if want.numel():
        top = max(top, float(want.abs().max()))
        off = (got - want).abs() - half * want.abs() - F32 * top
        assert float(off.max()) <= 0, f"{name}: off by {float((got - want).abs().max()):.3e} of {top:.3e}"


def formula(v, lengths=None):
    """(y, h_n, gradients by name, magnitudes of the terms of dt's and dt_bias'), row by
    row: what a row does not have is not in its sums."""
    names = ("x", "dt", "a_log", "b", "c", "d", "dt_bias", "z", "h0")
    leaves = [v[n].clone().requires_grad_() for n in names]
    x, dt, a_log, b, c, d, dt_bias, z, h0 = leaves
    T, B, H = x.shape

    def outputs(dt_in=None):
        ys, hs = [], []
        for r in range(B):
            n = T if lengths is None else int(lengths[r])
            row = slice(r, r + 1)
            y, h, _ = ref.scan(x[:n, row], dt[:n, row], a_log, b[:n, row], c[:n, row], d, dt_bias, z[:n, row], None,
                               h0[row], dt_in=None if dt_in is None else dt_in[:n, row])
            ys.append(torch.cat([y, torch.zeros(T - n, 1, H, dtype=y.dtype)]))
            hs.append(h)
        return torch.cat(ys, 1), torch.cat(hs)
    y, h = outputs()
    grads = dict(zip(NAMES, torch.autograd.grad((y, h), leaves, (v["dy"], v["dh_n"]))))
    apart = v["dt"].clone().requires_grad_()
    terms = sum(t.abs() for t in torch.autograd.grad(outputs(apart), (dt, apart), (v["dy"], v["dh_n"])))

    def most(t):
        t = t[torch.isfinite(t)]
        return float(t.max()) if t.numel() else 0.0
    return y, h, grads, {"ddt": most(terms), "ddt_bias": most(terms.sum((0, 1)))}


def check(ops, v, dtype, lengths=None):
    rows = ("x", "dt", "b", "c", "z", "dy")
    on = {k: t.to(DT[dtype] if k in rows else torch.float32).cuda() for k, t in v.items()}
    y, h, grads, tops = formula(v, lengths)
    ln = None if lengths is None else lengths.int().cuda()
    args = [on[k] for k in ("x", "dt", "a_log", "b", "c")]
    how = {"d": on["d"], "dt_bias": on["dt_bias"], "z": on["z"], "lengths": ln}
    got_y, got_h, states = ops.selscan_forward(*args, h0=on["h0"], states=True, **how)
    same(got_y, y, "y")
    same(got_h, h, "h_n")
    got = ops.selscan_backward(on["dy"], *args, states, dh_n=on["dh_n"], **how)
    for name in NAMES:
        same(got[name], grads[name], name, tops.get(name, 0.0))
    assert ops.status() == 0
    return y, grads


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 33, 38, 47])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_steps_that_are_not_there(ops, path, dtype, T, N):
    """A row's last input is infinite: its last state is, and no state that a decay meets."""
    v = inputs(T, 2, 12, N, dtype, [("x", (T - 1, 0, 5))])
    v["dh_n"][:] = 0
    _, g = check(ops, v, dtype)
    assert bool(torch.isfinite(g["da_log"]).all())
    if T > 3:
        v = inputs(T, 2, 12, N, dtype, [("x", (T - 3, 1, 5))])
        v["dh_n"][:] = 0
        _, g = check(ops, v, dtype, torch.tensor([T, T - 2]))
        assert bool(torch.isfinite(g["da_log"]).all())


STATES = [1, 2, 4, 5, 8, 11, 12, 16, 18, 24, 32, 33, 40, 64]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", STATES)
def test_states_that_are_not_there(ops, path, dtype, N):
    """An infinite x, and an infinite dy, at any number of states."""
    T, B, H = 45, 2, 8
    y, _ = check(ops, inputs(T, B, H, N, dtype, [("x", (9, 1, 3))]), dtype)
    assert not torch.isnan(y).any() and bool(torch.isinf(y[9:, 1, 3]).all())
    _, g = check(ops, inputs(T, B, H, N, dtype, [("dy", (30, 0, 5))]), dtype)
    assert bool(torch.isinf(g["dx"][:31, 0, 5]).all()) and not torch.isnan(g["dx"]).any()


@pytest.mark.parametrize("N", [4, 30])
@pytest.mark.parametrize("T", [1, 2, 3, 33, 47])
def test_steps_and_states_that_are_not_there(ops, path, T, N):
    test_steps_that_are_not_there(ops, path, "bf16", T, N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [1, 3, 4, 20, 63, 68])
@pytest.mark.parametrize("N", [4, 16, 32, 64])
def test_channels_that_are_not_there(ops, path, dtype, H, N):
    """An infinite b or c, whose gradients are sums over channels."""
    T, B = 45, 2
    n = N // 2
    _, g = check(ops, inputs(T, B, H, N, dtype, [("c", (30, 1, n))]), dtype)
    assert bool(torch.isinf(g["db"][:31, 1, n]).all()) and not torch.isnan(g["db"]).any()
    _, g = check(ops, inputs(T, B, H, N, dtype, [("b", (9, 0, n))]), dtype)
    assert bool(torch.isinf(g["dc"][9:, 0, n]).all()) and not torch.isnan(g["dc"]).any()


@pytest.mark.parametrize("T", [40, 700])
def test_an_infinite_state_outlasts_a_segment(ops, T):
    """States that decay far below fp32's range within a segment, and are infinite: kept
    infinite by every step's decay, so by the segment's too.  And their gradients."""
    v = inputs(T, 1, 8, 4, "f32", [("h0", (0, 3, 1))], slow=4.0)
    y, _ = check(ops, v, "f32")
    assert bool(torch.isinf(y[:, 0, 3]).all())
    _, g = check(ops, inputs(T, 1, 8, 4, "f32", [("dh_n", (0, 6, 2))], slow=4.0), "f32")
    assert bool(torch.isinf(g["dx"][:, 0, 6]).all()) and bool(torch.isinf(g["dh0"][0, 6, 2]))


@pytest.mark.parametrize("N", STATES)
def test_an_infinite_step_size(ops, path, N):
    """It forgets every state that exists, and makes it infinite."""
    v = inputs(45, 2, 8, N, "f32", [("dt", (9, 1, 3))])
    y, h, *_ = formula(v)
    on = {k: t.float().cuda() for k, t in v.items()}
    got = ops.selscan_forward(*(on[k] for k in ("x", "dt", "a_log", "b", "c")), h0=on["h0"], d=on["d"],
                              dt_bias=on["dt_bias"], z=on["z"])
    assert bool(torch.isinf(y[9:, 1, 3]).all()) and not torch.isnan(y).any()
    same(got[0], y, "y")
    same(got[1], h, "h_n")
