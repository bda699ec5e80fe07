"""Infinite logits and NaN in the gated linear recurrence on the GPU.  fp32 and the single
step: what the formulas say of them, exactly (sigmoid(-inf) is 0, so r = -inf holds a
state and i = -inf lets nothing in; a NaN reaches what the formulas make of it, forwards
and backwards).  bf16 sequences: logits stop at -42, and a NaN in i reaches its channel's
earlier gradients."""
import math

import pytest
import torch

from test_gpu_seq_ops import act8_values, close, ops, path, rec_backward, rec_forward, rec_inputs  # noqa: F401

pytestmark = pytest.mark.gpu

# whole rows, clusters, shares, segments; short sequences of many rows
SHAPES = [(96, 2, 66), (4111, 2, 72), (130, 500, 40), (9000, 1, 64), (9, 310, 131), (20, 250, 66)]


def cuda(*ts):
    return [t.cuda() for t in ts]


@pytest.mark.parametrize("T,B,H", SHAPES)
def test_closed_gates_hold_the_state(ops, path, T, B, H, dtype="f32"):  # noqa: F811
    """r = -inf from some step on: the state of before, to the bit, and no gradient to the
    inputs of those steps."""
    x, r, i, lam, h0 = rec_inputs(T, B, H, dtype, 51)
    lam[H // 2] = 3.0  # a channel that takes the general decay
    half = T // 32 * 16 if T >= 32 else T // 2  # where a warp of the tiled kernel starts
    r[half:] = -math.inf
    xd, rd, id_, ld, hd = cuda(x, r, i, lam, h0)
    y, h_n, st = ops.linrec_forward(xd, rd, id_, ld, h0=hd, states=True)
    _, h_half, _ = ops.linrec_forward(xd[:half], rd[:half], id_[:half], ld, h0=hd)
    close(h_half, h_n.cpu().double(), "h_n")  # (another length may be cut another way)
    if T < 9000:  # segments join their maps each in its own order
        assert torch.equal(y[half:], y[half:half + 1].expand(T - half, B, H))
    assert torch.equal(h_n.to(y.dtype), y[-1])
    dy = torch.randn(T, B, H, generator=torch.Generator().manual_seed(3)).to(x.dtype).cuda()
    dx, dr, di, dlam, dh0 = ops.linrec_backward(dy, xd, rd, id_, ld, st)
    top = float(dx.abs().max())
    assert float(dx[half:].abs().max()) <= 1e-17 * top  # 0 by the formulas
    assert not bool(dr[half:].any()) and not bool(di[half:].any())
    assert all(bool(torch.isfinite(t).all()) for t in (dx, dr, di, dlam, dh0))
    assert ops.status() == 0


@pytest.mark.parametrize("T,B,H", SHAPES)
def test_closed_inputs_let_nothing_in(ops, path, T, B, H, dtype="f32"):  # noqa: F811
    """i = -inf: the passes of inputs that are 0 there, however large they are."""
    x, r, i, lam, h0 = rec_inputs(T, B, H, dtype, 52)
    at = torch.rand(x.shape, generator=torch.Generator().manual_seed(5)) < 0.3
    i[at] = -math.inf
    zero, large = x.clone(), x.clone()
    zero[at], large[at] = 0, 1e30
    dy = torch.ones_like(x)
    rd, id_, ld, hd, dyd = cuda(r, i, lam, h0, dy)

    def passes(x):
        y, h_n, st = ops.linrec_forward(x, rd, id_, ld, h0=hd, states=True)
        return (y, h_n, st, *ops.linrec_backward(dyd, x, rd, id_, ld, st, dh_n=h_n))
    for a, b in zip(passes(zero.cuda()), passes(large.cuda())):
        assert torch.equal(a, b)
    assert ops.status() == 0


@pytest.mark.parametrize("T,B,H", SHAPES)
def test_bf16_logits_stop_at_42_below(ops, path, T, B, H):  # noqa: F811
    x, r, i, lam, h0 = rec_inputs(T, B, H, "bf16", 56)
    g = torch.Generator().manual_seed(8)
    for t in (r, i):
        t[torch.rand(x.shape, generator=g) < 0.1] = -math.inf
        t[torch.rand(x.shape, generator=g) < 0.1] = -60
    x[torch.isinf(i)] = 1e18  # lets in 0.6 of it
    xd, rd, id_, ld, hd = cuda(x, r, i, lam, h0)
    y, h_n, st = ops.linrec_forward(xd, rd, id_, ld, h0=hd, states=True)
    wide = [x.double(), r.double().clamp(min=-42), i.double().clamp(min=-42), lam.double()]
    ln = torch.full((B,), T)
    ry, rh, _ = rec_forward(*wide, 8.0, ln, h0.double())
    close(y, ry, "y")
    close(h_n, rh, "h_n")
    dy = torch.randn(T, B, H, generator=g).bfloat16()
    got = ops.linrec_backward(dy.cuda(), xd, rd, id_, ld, st)
    ref = rec_backward(dy.double(), *wide, st.cpu().double(), 8.0, ln, None)
    for name, p, q in zip(("dx", "dr", "di"), got, ref):
        close(p, q, name)
    close(got[4], ref[4], "dh0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H", [(150, 2, 66), (9, 310, 66)])
@pytest.mark.parametrize("which", [0, 1, 2], ids=["x", "r", "i"])
def test_nan_goes_where_the_formulas_take_it(ops, path, T, B, H, dtype, which):  # noqa: F811
    ins = rec_inputs(T, B, H, dtype, 53)
    t, b, h = T // 2, 1, 9
    ins[which][t, b, h] = math.nan
    x, r, i, lam, h0 = ins
    y, h_n, st = ops.linrec_forward(*cuda(x, r, i, lam), h0=h0.cuda(), states=True)
    wide = [v.double() for v in (x, r, i, lam)]
    ln = torch.full((B,), T)
    ry, rh, rst = rec_forward(*wide, 8.0, ln, h0.double())
    close(y, ry, "y")
    close(h_n, rh, "h_n")
    close(st, rst, "states")
    dy = torch.randn(T, B, H, generator=torch.Generator().manual_seed(6)).to(x.dtype)
    got = ops.linrec_backward(dy.cuda(), *cuda(x, r, i, lam), st)
    ref = rec_backward(dy.double(), *wide, st.cpu().double(), 8.0, ln, None)
    assert torch.equal(torch.isnan(got[3]).cpu(), torch.isnan(ref[3]))
    if dtype == "bf16" and which == 2:
        for p, q in zip(got[:3], ref):  # and the channel's earlier steps
            also = torch.isnan(p).cpu() & ~torch.isnan(q)
            assert not bool((torch.isnan(q) & ~torch.isnan(p).cpu()).any())
            also[:t, b, h] = False
            assert not bool(also.any())
        return
    for name, p, q in zip(("dx", "dr", "di"), got, ref):
        close(p, q, name)
    close(got[4], ref[4], "dh0")


def test_step_with_closed_gates(ops, path):  # noqa: F811
    for dtype in ("f32", "bf16"):
        x, r, i, lam, h0 = rec_inputs(1, 5, 64, dtype, 54)
        x[0, 1] = 1e30
        r[0, 0] = -math.inf
        i[0, 1] = -math.inf
        xd, rd, id_, ld, state = cuda(x[0], r[0], i[0], lam, h0)
        y = ops.linrec_step(xd, rd, id_, ld, state)
        assert torch.equal(state[0].cpu(), h0[0]) and torch.equal(y[0], state[0].to(y.dtype))
        ref, _, _ = rec_forward(*(t.double() for t in (x, r, i, lam)), 8.0, torch.full((5,), 1), h0.double())
        close(y[1:2], ref[0, 1:2], "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H", [(96, 2, 64), (9, 310, 64), (9000, 1, 64)])
def test_large_logits_from_8_bits(ops, path, T, B, H, dtype):  # noqa: F811
    """Blocks whose logits reach +-1e30: gates of 0 and 1 exactly."""
    x, r, i, lam, h0 = rec_inputs(T, B, H, dtype, 55)
    r[::2], i[1::2] = r[::2] * 1e30, i[1::2] * 1e30
    xd, rd, id_, ld, hd = cuda(x, r, i, lam, h0)
    _, _, st = ops.linrec_forward(xd, rd, id_, ld, h0=hd, states=True)
    saved = [ops.act8_pack(t) for t in (xd, rd, id_)]
    dy = torch.randn(T, B, H, generator=torch.Generator().manual_seed(7)).to(x.dtype)
    got = ops.linrec_backward(dy.cuda(), *saved, ld, st)
    wide = [act8_values(a.cpu(), b.cpu()) for a, b in saved]
    ref = rec_backward(dy.double(), *wide, lam.double(), st.cpu().double(), 8.0, torch.full((B,), T), None)
    for name, p, q in zip(("dx", "dr", "di"), got, ref):
        close(p, q, name)
    close(got[4], ref[4], "dh0")
