"""GPU parity of the gated linear recurrence with gates and decays of any size, in
every form of its kernels: short sequences of many rows, shares of the tiles,
clusters and segments, from full types and from 8 bits.  Rates between "remembers
all" and "forgets at once" stand beside one another in a row, so every warp takes
the general form of the decay with its ceilings on the logits.  Tolerances as in
test_gpu_seq_ops.py.
"""
import pytest
import torch

from recurrent_cell_unroll_gb300 import binding
from test_gpu_seq_ops import DT, check_rec, ops, path, rec_inputs  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def wide_inputs(T, B, H, dtype, batch_first, rates):
    """Logits from -30 to 30 beside decay parameters from -30 to 30, or up to where
    fp32 ends."""
    g = torch.Generator().manual_seed(T + B + H)
    shape = (B, T, H) if batch_first else (T, B, H)
    x = torch.randn(shape, generator=g)
    r, i = (torch.rand(shape, generator=g) * 60 - 30 for _ in range(2))
    lam = torch.linspace(-30, 30, H) if rates == "any" else torch.exp2(torch.linspace(-4, 120, H))
    return [t.to(DT[dtype]) for t in (x, r, i)] + [lam, torch.randn(B, H, generator=g)]


@pytest.mark.parametrize("act", [False, True], ids=["full", "8-bits"])
@pytest.mark.parametrize("rates", ["any", "fast"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,batch_first,varied", [
    (1, 480, 33, False, False), (11, 300, 131, False, True), (14, 310, 132, True, True),
    (14, 240, 192, False, False), (40, 470, 33, False, True),            # short, many rows
    (130, 500, 40, False, True), (200, 131, 300, True, False),           # shares
    (4111, 2, 72, False, True), (9000, 1, 64, False, False)])            # clusters, segments
def test_linrec_any_decay(request, ops, path, T, B, H, batch_first, varied, dtype, rates, act):  # noqa: F811
    if T == 9000 and rates == "any":
        # lam = -19.5: a is 1 - 1.3e-8, which an fp32 product of decays takes for 1.  One
        # multiplication and addition a step in fp32 is off by as much (1.08e-4 of 1.96).
        request.applymarker(pytest.mark.xfail(strict=True, reason="a decay below the last bit of 1"))
    lengths = [(7 * b + T) % (T + 1) for b in range(B)] if varied else None
    check_rec(ops, T, B, H, dtype, batch_first, lengths, act=act,
              inputs=wide_inputs(T, B, H, dtype, batch_first, rates))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H", [(20, 250, 131), (3, 500, 64), (700, 3, 65)])
def test_linrec_one_fast_channel(ops, path, T, B, H, dtype):  # noqa: F811
    """Channels of ordinary decays beside one that forgets at once."""
    x, r, i, lam, h0 = rec_inputs(T, B, H, dtype, 41)
    lam[H // 2] = 3.0
    check_rec(ops, T, B, H, dtype, inputs=(x, r, i, lam, h0))
    check_rec(ops, T, B, H, dtype, inputs=(x, r, i, lam, h0), act=True)


def test_linrec_step_any_decay(ops, path):  # noqa: F811
    """A step is the forward of one step, whatever its gates."""
    for dtype in ("f32", "bf16"):
        x, r, i, lam, h0 = (t.cuda() for t in wide_inputs(1, 9, 64, dtype, False, "any"))
        y, h_n, _ = ops.linrec_forward(x, r, i, lam, h0=h0)
        state = h0.clone()
        out = ops.linrec_step(x[0], r[0], i[0], lam, state)
        scale = float(h_n.abs().max())
        assert float((state - h_n).abs().max()) <= 2e-5 * scale
        half = 2.0 ** -8 if dtype == "bf16" else 0.0
        assert bool(((out - y[0]).abs() <= half * y[0].abs() + 2e-5 * scale).all())
    assert ops.status() == binding.RCU_OK
