"""GPU parity of the sequence operators (gated linear recurrence, layer norm,
8-bit activation checkpoints) against plain 64-bit implementations, at the
sizes, masks, strides and values where they can go wrong.

Tolerances: an fp32 result is within F32 of its tensor's largest magnitude.
Each gate carries a few roundings (an exponential of base 2 whose argument is
rounded at |v| <= 2^5: 2^-24 * 2^5 / 2 ~ 1e-6), and a sum over the steps that a
state remembers, or over rows, at most a few tens of that.  A bf16 result is
rounded once more: half a unit in its last place, 2^-8 of the value.
"""
import itertools
import math

import pytest
import torch

from recurrent_cell_unroll_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16_HALF = 2e-5, 2.0 ** -8
CHUNK, BLOCK = 64, 64
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


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


def close(got, ref, name, scale=None):
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    half = BF16_HALF if got.dtype == torch.bfloat16 else 0.0
    got = got.detach().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{name}: NaN in other places"
    got, ref = torch.nan_to_num(got, nan=0.0), torch.nan_to_num(ref, nan=0.0)
    top = float(ref.abs().max()) if scale is None else scale
    off = (got - ref).abs() - half * ref.abs() - F32 * top
    assert float(off.max()) <= 0, f"{name}: off by {float((got - ref).abs().max()):.3e} of {top:.3e}"


# --------------------------------------------------------------------------- 64-bit definitions

def rec_gates(x, r, i, lam, c):
    sp = torch.logaddexp(lam, torch.zeros_like(lam))
    s, g = torch.sigmoid(r), torch.sigmoid(i)
    em1 = torch.expm1(-c * sp * s)
    return s, g, em1, torch.sqrt(-em1 * (2 + em1))


def rec_forward(x, r, i, lam, c, lengths, h0):
    """Time-major, fp64, one step after another."""
    T, B, H = x.shape
    s, g, em1, beta = rec_gates(x, r, i, lam, c)
    h = torch.zeros(B, H, dtype=torch.float64) if h0 is None else h0
    y, states = torch.zeros(T, B, H, dtype=torch.float64), []
    for t in range(T):
        if t % CHUNK == 0:
            states.append(h)
        on = (t < lengths)[:, None]
        h = torch.where(on, h + em1[t] * h + beta[t] * g[t] * x[t], h)
        y[t] = torch.where(on, h, torch.zeros_like(h))
    return y, h, torch.stack(states) if states else torch.zeros(0, B, H, dtype=torch.float64)


def rec_backward(dy, x, r, i, lam, states, c, lengths, dh_n):
    T, B, H = x.shape
    s, g, em1, beta = rec_gates(x, r, i, lam, c)
    before = torch.zeros(T, B, H, dtype=torch.float64)
    for t in range(T):
        h = states[t // CHUNK] if t % CHUNK == 0 else h
        before[t] = h
        h = h + em1[t] * h + beta[t] * g[t] * x[t]
    e = torch.zeros(B, H, dtype=torch.float64) if dh_n is None else dh_n
    sp = torch.logaddexp(lam, torch.zeros_like(lam))
    dx, dr, di = (torch.zeros(T, B, H, dtype=torch.float64) for _ in range(3))
    dsp = torch.zeros(B, H, dtype=torch.float64)
    for t in reversed(range(T)):
        on = (t < lengths)[:, None]
        full = e + dy[t]
        a = 1 + em1[t]
        # d sqrt(1 - a^2) / d log a = -a^2 / beta: times s it has a limit where beta is 0
        s_beta = torch.where(beta[t] > 0, s[t] / beta[t], torch.zeros_like(full))
        dlog_s = full * (a * before[t] * s[t] - a * a * g[t] * x[t] * s_beta)
        zero = torch.zeros_like(full)
        dx[t] = torch.where(on, full * beta[t] * g[t], zero)
        di[t] = torch.where(on, full * beta[t] * x[t] * g[t] * (1 - g[t]), zero)
        dr[t] = torch.where(on, -c * sp * dlog_s * (1 - s[t]), zero)
        dsp = dsp + torch.where(on, -c * dlog_s, zero)
        e = torch.where(on, a * full, e)
    return dx, dr, di, (dsp * torch.sigmoid(lam)).sum(0), e


def ln_forward(x, weight, bias, eps):
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = 1 / torch.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[..., None]
    if weight is not None:
        y = y * weight
    return (y + bias if bias is not None else y), mean, rstd


def ln_backward(dy, u, mean, rstd, weight, dsum):
    xh = (u - mean[..., None]) * rstd[..., None]
    q = dy if weight is None else dy * weight
    du = rstd[..., None] * (q - q.mean(-1, keepdim=True) - xh * (q * xh).mean(-1, keepdim=True))
    lead = tuple(range(dy.dim() - 1))
    return du + (0 if dsum is None else dsum), (dy * xh).sum(lead), dy.sum(lead)


def act8(v):
    """Codes and exponents, value by value."""
    n = v.shape[-1]
    codes = torch.zeros(v.shape, dtype=torch.int8)
    exps = torch.zeros(*v.shape[:-1], -(-n // BLOCK), dtype=torch.int8)
    for row in itertools.product(*map(range, v.shape[:-1])):
        for k in range(exps.shape[-1]):
            part = [float(f) for f in v[row][k * BLOCK:(k + 1) * BLOCK]]
            top = max([abs(f) for f in part if math.isfinite(f)], default=0.0)
            e = -126
            while 127 * 2.0 ** e < top and e < 121:  # 64 * 2^122 would be infinite
                e += 1
            exps[row][k] = e
            for j, f in enumerate(part):
                codes[row][k * BLOCK + j] = \
                    max(-127, min(127, round(f / 2.0 ** e))) if math.isfinite(f) else -128
    return codes, exps


def act8_values(codes, exps):
    at = torch.arange(codes.shape[-1]) // BLOCK
    v = codes.double() * torch.exp2(exps.double())[..., at]
    return torch.where(codes == -128, torch.full_like(v, math.nan), v)


# --------------------------------------------------------------------------- gated linear recurrence

def rec_inputs(T, B, H, dtype, seed=0, batch_first=False, std=1.0):
    g = torch.Generator().manual_seed(seed)
    shape = (B, T, H) if batch_first else (T, B, H)
    x, r, i = (torch.randn(shape, generator=g) * std for _ in range(3))
    top = 0.9 + 0.099 * torch.rand(H, generator=g)
    lam = torch.log(torch.expm1(-torch.log(top) / 8.0))
    return [t.to(DT[dtype]) for t in (x, r, i)] + [lam, torch.randn(B, H, generator=g) * 0.5]


def check_rec(ops, T, B, H, dtype, batch_first=False, lengths=None, use_h0=True, c=8.0, seed=0,
              act=False, inputs=None, wide=False):
    x, r, i, lam, h0 = inputs or rec_inputs(T, B, H, dtype, seed, batch_first)
    g = torch.Generator().manual_seed(seed + 100)
    dy = torch.randn(x.shape, generator=g).to(DT[dtype])
    dh_n = torch.randn(B, H, generator=g)
    h0 = h0 if use_h0 else None
    ln = torch.full((B,), T) if lengths is None else torch.tensor(lengths)

    def tf(t):
        return t.transpose(0, 1) if batch_first else t

    def dev(t):
        if t is None:
            return None
        if wide and t.dim() == 3:  # a slice of a wider tensor, not 16-byte aligned
            big = torch.zeros(*t.shape[:2], 3 * H + 5, dtype=t.dtype, device="cuda")
            big[..., H + 1:2 * H + 1] = t.cuda()
            return big[..., H + 1:2 * H + 1]
        return t.cuda()
    dl = None if lengths is None else ln.int().cuda()
    xd, rd, id_, dyd = (dev(t) for t in (x, r, i, dy))
    y, h_n, states = ops.linrec_forward(xd, rd, id_, lam.cuda(), c=c, lengths=dl, h0=dev(h0),
                                        batch_first=batch_first, states=True)
    wide_in = [torch.nan_to_num(tf(t).double()) if lengths is not None else tf(t).double()
               for t in (x, r, i)]
    ry, rh, rst = rec_forward(*wide_in, lam.double(), c, ln, None if h0 is None else h0.double())
    close(tf(y), ry, "y")
    close(h_n, rh, "h_n")
    close(states, rst, "states")
    saved = (xd, rd, id_)
    if act:
        saved = [ops.act8_pack(t) for t in saved]
        wide_in = [tf(act8_values(a.cpu(), b.cpu())) for a, b in saved]
    got = ops.linrec_backward(dyd, *saved, lam.cuda(), states, c=c, lengths=dl, dh_n=dev(dh_n),
                              batch_first=batch_first)
    ref = rec_backward(torch.nan_to_num(tf(dy).double()), *wide_in, lam.double(),
                       states.cpu().double(), c, ln, dh_n.double())
    assert ops.status() == 0
    # dr sums two terms that can cancel: their scale is that of the gradient itself
    for name, a, b in zip(("dx", "dr", "di"), got, ref):
        close(tf(a), b, name)
    close(got[3], ref[3], "dlam", scale=max(float(ref[3].abs().max()), dlam_scale(ref, wide_in)))
    close(got[4], ref[4], "dh0")


def dlam_scale(ref, ins):
    """dlambda sums terms of both signs: rounding goes by the terms' root mean
    square times the root of their number."""
    dr, r = ref[1], ins[1]
    terms = dr / (1 - torch.sigmoid(r)).clamp(min=1e-6)  # = K dlog_s, the summand but for a factor < 1
    n = terms.shape[0] * terms.shape[1]
    return float(terms.square().mean().sqrt()) * math.sqrt(n) if n else 0.0


REC_SIZES = [
    (1, 1, 1), (1, 3, 8), (2, 1, 33), (63, 2, 64), (64, 1, 65), (65, 3, 32), (80, 1, 256),
    (127, 2, 100), (128, 4, 128), (129, 1, 31), (200, 5, 96), (513, 2, 72), (1000, 1, 200),
    (2100, 1, 64), (300, 17, 40),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H", REC_SIZES)
def test_linrec_sizes(ops, path, T, B, H, dtype):
    check_rec(ops, T, B, H, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H", [(65, 3, 32), (130, 2, 200), (300, 4, 65)])
def test_linrec_batch_first(ops, path, T, B, H, dtype):
    check_rec(ops, T, B, H, dtype, batch_first=True)


@pytest.mark.parametrize("batch_first", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linrec_lengths(ops, path, dtype, batch_first):
    """Lengths of zero, one, the chunk's edges and T; NaN where no step is."""
    T, lengths = 200, [0, 1, 63, 64, 65, 128, 199, 200, 7, 130]
    B, H = len(lengths), 72
    x, r, i, lam, h0 = rec_inputs(T, B, H, dtype, 3, batch_first)
    for t in (x, r, i):
        v = t if batch_first else t.transpose(0, 1)
        for b, n in enumerate(lengths):
            v[b, n:] = math.nan
    check_rec(ops, T, B, H, dtype, batch_first, lengths, inputs=(x, r, i, lam, h0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,batch_first,act,lengths", [
    (1, 320, 33, False, False, False), (4, 170, 130, False, False, True),
    (5, 330, 64, True, True, True), (19, 160, 131, False, True, False), (20, 110, 192, True, False, True),
    (21, 110, 192, False, False, False), (13, 170, 131, False, False, True), (48, 320, 33, False, True, True),
    (49, 310, 33, True, False, False)])
def test_linrec_short_sequences_of_many_rows(ops, path, dtype, T, B, H, batch_first, act, lengths):
    ln = [(7 * b) % (T + 1) for b in range(B)] if lengths else None
    check_rec(ops, T, B, H, dtype, batch_first, ln, act=act)
    if T == 4:
        check_rec(ops, T, B, H, dtype, wide=True)


def test_linrec_all_rows_empty(ops, path):
    check_rec(ops, 130, 3, 40, "bf16", lengths=[0, 0, 0])


def test_linrec_nan_dy_past_the_end(ops, path):
    T, B, H = 100, 2, 64
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, "f32", 4))
    ln = torch.tensor([40, 100], dtype=torch.int32, device="cuda")
    _, _, st = ops.linrec_forward(x, r, i, lam, lengths=ln, h0=h0, states=True)
    dy = torch.randn(T, B, H, device="cuda")
    ref = ops.linrec_backward(dy, x, r, i, lam, st, lengths=ln)
    dy[40:, 0] = math.nan
    got = ops.linrec_backward(dy, x, r, i, lam, st, lengths=ln)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linrec_slices_of_wider_tensors(ops, path, dtype):
    check_rec(ops, 150, 3, 64, dtype, wide=True)
    check_rec(ops, 70, 2, 40, dtype, wide=True, batch_first=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,batch_first,lengths", [
    (1, 500, 33, False, False), (3, 240, 130, True, True), (8, 470, 64, False, True),
    (9, 240, 67, True, False), (31, 160, 200, False, True), (32, 480, 30, True, True),
    (33, 480, 30, False, False), (64, 460, 31, True, True), (20, 240, 67, False, False),
    (21, 240, 67, False, True), (32, 500, 64, False, False)])
def test_linrec_forward_of_short_sequences(ops, path, dtype, T, B, H, batch_first, lengths):
    ln = [(5 * b) % (T + 1) for b in range(B)] if lengths else None
    check_rec(ops, T, B, H, dtype, batch_first, ln)
    if T == 9:
        check_rec(ops, T, B, H, dtype, use_h0=False, wide=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H", [(130, 3, 77), (65, 400, 75)])
def test_linrec_inputs_that_lie_differently(ops, path, dtype, T, B, H):
    """Rows at other offsets and strides than their neighbours': the same bits."""
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, dtype, 9))

    def moved(t, width, at):
        big = torch.zeros(*t.shape[:2], width, dtype=t.dtype, device="cuda")
        big[..., at:at + H] = t
        return big[..., at:at + H]

    def passes(x, r, i, dy):
        y, h_n, st = ops.linrec_forward(x, r, i, lam, h0=h0, states=True)
        return (y, h_n, *ops.linrec_backward(dy, x, r, i, lam, st, dh_n=h_n))
    want = passes(x, r, i, x)
    got = passes(x, moved(r, H + 4, 3), moved(i, 2 * H, 1), moved(x, H + 1, 1))
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_linrec_without_h0(ops, path):
    check_rec(ops, 90, 2, 64, "f32", use_h0=False)


@pytest.mark.parametrize("c", [0.5, 8.0, 40.0])
def test_linrec_decay_constants(ops, path, c):
    check_rec(ops, 100, 2, 64, "f32", c=c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,batch_first,lengths",
                         [(130, 2, 64, False, None), (100, 3, 130, True, [100, 0, 65]),
                          (65, 1, 33, False, None), (513, 2, 192, False, [513, 300])])
def test_linrec_backward_from_8_bits(ops, path, dtype, T, B, H, batch_first, lengths):
    check_rec(ops, T, B, H, dtype, batch_first, lengths, act=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linrec_long_sequence_of_few_channels(ops, path, dtype):
    """Time split over the GPU: more than one round of the split, and its seams."""
    check_rec(ops, 9000, 1, 40, dtype)
    check_rec(ops, 4111, 2, 33, dtype, lengths=[4111, 2049])


@pytest.mark.parametrize("T,B,H,lengths", [(20000, 1, 33, None), (12345, 2, 40, [12345, 9000]),
                                           (16000, 1, 16, [0])])
def test_linrec_segments(ops, path, T, B, H, lengths):
    """So few channels that the sequence runs in segments (two launches a pass)."""
    check_rec(ops, T, B, H, "bf16", lengths=lengths)
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, "bf16"))
    _, _, st = ops.linrec_forward(x, r, i, lam, h0=h0, states=True)
    assert ops.launch_count() == 2
    ops.linrec_backward(x, x, r, i, lam, st)
    assert ops.launch_count() == 3


@pytest.mark.parametrize("dtype,T,B,H,batch_first,act,lengths",
                         [("bf16", 130, 500, 40, False, False, None),
                          ("bf16", 200, 131, 300, True, False, "mixed"),
                          ("f32", 130, 350, 64, False, True, "mixed"),
                          ("bf16", 321, 160, 200, False, True, None),
                          ("f32", 70, 600, 33, True, False, "mixed")])
def test_linrec_shares(ops, path, dtype, T, B, H, batch_first, act, lengths):
    """More rows than blocks and no multiple of them: rows that two blocks have a part of."""
    if lengths:
        g = torch.Generator().manual_seed(B)
        lengths = torch.randint(0, T + 1, (B,), generator=g).tolist()
    check_rec(ops, T, B, H, dtype, batch_first, lengths, act=act)


def test_linrec_shares_in_a_graph(ops, path):
    """Replays start from flags of their own, and give the same bits each time."""
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(130, 500, 40, "bf16", 31))

    def passes():
        y, h_n, st = ops.linrec_forward(x, r, i, lam, h0=h0, states=True)
        return (y, h_n, *ops.linrec_backward(y, x, r, i, lam, st, dh_n=h_n))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = passes()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = passes()
    for _ in range(3):
        for t in held:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want))
    assert ops.status() == 0


def test_linrec_nan_codes(ops, path):
    """A code that is not a number reaches what its value enters, and no more."""
    T, B, H = 70, 1, 64
    for dtype in ("f32", "bf16"):
        x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, dtype, 21))
        _, _, st = ops.linrec_forward(x, r, i, lam, h0=h0, states=True)
        dy = torch.ones_like(x)
        saved = [ops.act8_pack(t) for t in (x, r, i)]
        clean = ops.linrec_backward(dy, *saved, lam, st)
        for k in range(3):
            codes = saved[k][0].clone()
            codes[66, 0, 5] = -128
            bad = list(saved)
            bad[k] = (codes, saved[k][1])
            got = ops.linrec_backward(dy, *bad, lam, st)
            wide = [act8_values(a.cpu(), b.cpu()) for a, b in bad]
            ref = rec_backward(dy.cpu().double(), *wide, lam.cpu().double(), st.cpu().double(), 8.0,
                               torch.tensor([T]), None)
            for a, b, c in zip(got[:3], ref, clean):
                assert torch.equal(torch.isnan(a).cpu(), torch.isnan(b))
                same = ~torch.isnan(a)
                assert torch.equal(a[same], c[same])


def test_linrec_extreme_gates(ops, path):
    """Logits from -90 to 90 and infinite ones, decay parameters from -30 to 30:
    decays of exactly 0 and 1, input scales of 0, no NaN anywhere."""
    T, B, H = 96, 2, 64
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, B, H, generator=g)
    r, i = (torch.rand(T, B, H, generator=g) * 60 - 30 for _ in range(2))
    lam = torch.linspace(-30, 30, H)
    h0 = torch.randn(B, H, generator=g)
    check_rec(ops, T, B, H, "f32", inputs=(x, r, i, lam, h0))
    check_rec(ops, T, B, H, "bf16", inputs=(*(t.bfloat16() for t in (x, r, i)), lam, h0))
    # decay rates up to where fp32 ends: the gate's ceiling in every binade
    lam2 = torch.exp2(torch.linspace(-4, 120, H))
    check_rec(ops, T, B, H, "bf16", inputs=(*(t.bfloat16() for t in (x, r, i)), lam2, h0))
    check_rec(ops, T, B, H, "f32", inputs=(x, r, i, lam2, h0))
    vals = torch.tensor([-math.inf, -90.0, -50.0, 50.0, 90.0, math.inf])
    r = vals[torch.randint(0, 6, (T, B, H), generator=g)]
    i = vals[torch.randint(0, 6, (T, B, H), generator=g)]
    xd, rd, id_, ld, hd = (t.cuda() for t in (x, r, i, lam, h0))
    y, h_n, st = ops.linrec_forward(xd, rd, id_, ld, h0=hd, states=True)
    dy = torch.randn(T, B, H, generator=g)
    got = ops.linrec_backward(dy.cuda(), xd, rd, id_, ld, st)
    ref, _, _ = rec_forward(*(t.double() for t in (x, r, i, lam)), 8.0, torch.full((B,), T),
                            h0.double())
    close(y, ref, "y")
    for t in (y, h_n, *got):
        assert bool(torch.isfinite(t).all())


@pytest.mark.parametrize("dtype,T,B,H", [("f32", 96, 2, 128), ("bf16", 96, 2, 128), ("bf16", 14, 300, 131),
                                         ("f32", 14, 310, 33), ("bf16", 9000, 1, 64)])
def test_linrec_wide_gates_from_8_bits(ops, path, dtype, T, B, H):
    """Steps whose blocks hold logits beyond the gates' limits between steps without."""
    x, r, i, lam, h0 = rec_inputs(T, B, H, dtype, 10)
    r[::3] *= 60
    i[1::4] *= 60
    check_rec(ops, T, B, H, dtype, inputs=(x, r, i, lam, h0), act=True)


def test_linrec_nan_stays_in_its_row_and_channel(ops, path):
    T, B, H = 150, 2, 64
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, "f32", 5))
    for t in (x, r, i):
        y0, _, _ = ops.linrec_forward(x, r, i, lam, h0=h0)
        keep = t[70, 1, 9].clone()
        t[70, 1, 9] = math.nan
        y, h_n, _ = ops.linrec_forward(x, r, i, lam, h0=h0)
        t[70, 1, 9] = keep
        bad = torch.isnan(y)
        assert bool(bad[70:, 1, 9].all()) and int(bad.sum()) == T - 70
        assert torch.equal(y[~bad], y0[~bad])


def test_linrec_lengths_out_of_range_are_reported(ops):
    T, B, H = 70, 3, 32
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, "f32", 6))
    ln = torch.tensor([-3, 71, 20], dtype=torch.int32, device="cuda")
    y, _, _ = ops.linrec_forward(x, r, i, lam, lengths=ln, h0=h0)
    assert ops.status() == binding.RCU_ERR_LENGTHS
    assert ops.status() == 0
    ok = torch.tensor([0, 70, 20], dtype=torch.int32, device="cuda")
    z, _, _ = ops.linrec_forward(x, r, i, lam, lengths=ok, h0=h0)
    assert torch.equal(y, z) and ops.status() == 0


def test_linrec_after_an_unread_report(ops):
    """A length out of range that nobody has asked about yet ends no later call's waits."""
    T, B, H = 4097, 3, 192
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, "bf16", 7))

    def passes():
        y, _, st = ops.linrec_forward(x, r, i, lam, h0=h0, states=True)
        return (y, *ops.linrec_backward(y, x, r, i, lam, st))
    want = passes()
    assert ops.status() == 0
    ops.linrec_forward(x, r, i, lam, lengths=torch.full((B,), T + 1, dtype=torch.int32, device="cuda"))
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(passes(), want))
    assert ops.status() == binding.RCU_ERR_LENGTHS


def test_linrec_empty(ops):
    x = torch.empty(0, 2, 8, device="cuda")
    lam, h0 = torch.zeros(8, device="cuda"), torch.randn(2, 8, device="cuda")
    y, h_n, st = ops.linrec_forward(x, x, x, lam, h0=h0, states=True)
    assert y.shape == (0, 2, 8) and st.shape == (0, 2, 8) and torch.equal(h_n, h0)
    _, h_n, _ = ops.linrec_forward(x, x, x, lam)
    assert not bool(h_n.any())
    *_, dlam, dh0 = ops.linrec_backward(x, x, x, x, lam, st, dh_n=h0)
    assert torch.equal(dh0, h0) and not bool(dlam.any())
    x = torch.empty(3, 0, 8, device="cuda")
    y, h_n, _ = ops.linrec_forward(x, x, x, lam)
    assert y.shape == (3, 0, 8) and h_n.shape == (0, 8)
    assert ops.linrec_step(x[0], x[0], x[0], lam, torch.empty(4, 8, device="cuda")).shape == (0, 8)


def test_linrec_is_reproducible(ops, path):
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(3000, 3, 96, "bf16", 7))
    a = ops.linrec_forward(x, r, i, lam, h0=h0, states=True)
    b = ops.linrec_forward(x, r, i, lam, h0=h0, states=True)
    dy = torch.randn_like(x)
    c = ops.linrec_backward(dy, x, r, i, lam, a[2])
    d = ops.linrec_backward(dy, x, r, i, lam, a[2])
    for p, q in zip((*a, *c), (*b, *d)):
        assert torch.equal(p, q)


def test_linrec_gradient_against_differences(ops):
    """Central differences of the 64-bit forward, at random places of every input."""
    T, B, H, c = 70, 2, 36, 8.0
    x, r, i, lam, h0 = rec_inputs(T, B, H, "f32", 9)
    g = torch.Generator().manual_seed(10)
    dy, dh_n = torch.randn(T, B, H, generator=g), torch.randn(B, H, generator=g)
    ln = torch.tensor([70, 66])
    d = [t.cuda() for t in (x, r, i, lam)]
    _, _, st = ops.linrec_forward(*d, lengths=ln.int().cuda(), h0=h0.cuda(), states=True)
    got = ops.linrec_backward(dy.cuda(), *d, st, lengths=ln.int().cuda(), dh_n=dh_n.cuda())
    ins = [t.double() for t in (x, r, i, lam, h0)]

    def loss():
        y, h, _ = rec_forward(ins[0], ins[1], ins[2], ins[3], c, ln, ins[4])
        return float((y * dy.double()).sum() + (h * dh_n.double()).sum())
    for k, grad in enumerate(got):
        flat = ins[k].view(-1)
        top = float(grad.abs().max())
        for at in torch.randint(0, flat.numel(), (12,), generator=g).tolist():
            keep, step = float(flat[at]), 1e-5
            flat[at] = keep + step
            up = loss()
            flat[at] = keep - step
            down = loss()
            flat[at] = keep
            # the difference itself is good to step^2 and 64-bit rounding / step: 1e-8 here
            assert abs((up - down) / (2 * step) - float(grad.view(-1)[at])) <= F32 * top + 1e-7, (k, at)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H", [(1, 1), (1, 256), (3, 33), (5, 100), (64, 128), (200, 72)])
def test_linrec_step(ops, path, B, H, dtype):
    x, r, i, lam, _ = rec_inputs(1, B, H, dtype, 11)
    x, r, i = x[0], r[0], i[0]
    g = torch.Generator().manual_seed(12)
    slots = 2 * B + 1
    state = torch.randn(slots, H, generator=g)
    slot = torch.randperm(slots, generator=g)[:B].int()
    if B > 2:
        slot[1] = -1
    sd = state.cuda()
    y = ops.linrec_step(x.cuda(), r.cuda(), i.cuda(), lam.cuda(), sd, slot=slot.cuda())
    ref, rst = torch.zeros(B, H, dtype=torch.float64), state.double()
    for b, at in enumerate(slot.tolist()):
        if at >= 0:
            one = [t[b:b + 1][None].double() for t in (x, r, i)]
            out, h, _ = rec_forward(*one, lam.double(), 8.0, torch.tensor([1]),
                                    state[at:at + 1].double())
            ref[b], rst[at] = out[0, 0], h[0]
    assert ops.status() == 0
    close(y, ref, "y")
    close(sd, rst, "state")
    untouched = torch.ones(slots, dtype=torch.bool)
    untouched[slot[slot >= 0].long()] = False
    assert torch.equal(sd.cpu()[untouched], state[untouched])


def test_linrec_step_slots_out_of_range(ops):
    B, H = 4, 32
    x = torch.randn(B, H, device="cuda")
    lam, state = torch.zeros(H, device="cuda"), torch.randn(3, H, device="cuda")
    slot = torch.tensor([2, 3, -2, 0], dtype=torch.int32, device="cuda")
    keep = state.clone()
    y = ops.linrec_step(x, x, x, lam, state, slot=slot)
    assert ops.status() == binding.RCU_ERR_SLOTS
    assert not bool(y[1:3].any()) and bool(y[0].any()) and torch.equal(state[1], keep[1])


def test_linrec_step_follows_the_forward(ops):
    """Prefill, then tokens one by one: the same states as one long forward."""
    T, B, H = 100, 3, 64
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, "f32", 13))
    y, h_n, _ = ops.linrec_forward(x, r, i, lam, h0=h0)
    _, state, _ = ops.linrec_forward(x[:90], r[:90], i[:90], lam, h0=h0)
    for t in range(90, T):
        out = ops.linrec_step(x[t], r[t], i[t], lam, state)
        close(out, y[t].cpu().double(), "y")
    close(state, h_n.cpu().double(), "state")


# --------------------------------------------------------------------------- layer norm

LN_SIZES = [(1, 1), (3, 2), (1, 7), (50, 200), (5, 31), (4, 64), (3, 100), (7, 257), (2, 1000),
            (300, 128), (33, 1024), (5, 2050), (9, 4096), (2, 5000), (3, 8192), (2, 16384),
            (1, 40001)]


def ln_inputs(rows, n, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g) * (0.5 + torch.rand(n, generator=g)) + 0.3
    rest = [torch.randn(rows, n, generator=g) for _ in range(3)]
    w, b = 1 + 0.1 * torch.randn(n, generator=g), 0.1 * torch.randn(n, generator=g)
    return [t.to(DT[dtype]) for t in (x, *rest)] + [w, b]


def check_ln(ops, rows, n, dtype, residual, affine=True, act=False, eps=1e-5, wide=False, seed=0):
    x, res, dy, dsum, w, b = ln_inputs(rows, n, dtype, seed)
    if not affine:
        w = b = None

    def dev(t):
        if t is None:
            return None
        if wide and t.dim() == 2:
            big = torch.zeros(rows, 2 * n + 3, dtype=t.dtype, device="cuda")
            big[:, n + 1:2 * n + 1] = t.cuda()
            return big[:, n + 1:2 * n + 1]
        return t.cuda()
    out = ops.layernorm_forward(dev(x), dev(w), dev(b), eps=eps, residual=dev(res) if residual else None)
    u = x
    if residual:
        u = (x.float() + res.float()).to(x.dtype)
        assert torch.equal(out[1].cpu(), u)
    wd, bd = (None if t is None else t.double() for t in (w, b))
    y, mean, rstd = ln_forward(u.double(), wd, bd, eps)
    close(out[0], y, "y")
    close(out[-2], mean, "mean", scale=float(u.double().abs().max()))
    close(out[-1], rstd, "rstd")
    ud = dev(u)
    saved, uw = ud, u.double()
    if act:
        saved = ops.act8_pack(ud)
        uw = act8_values(saved[0].cpu(), saved[1].cpu())
    du, dw, db = ops.layernorm_backward(dev(dy), saved, out[-2], out[-1], dev(w),
                                        dsum=dev(dsum) if residual else None)
    ref = ln_backward(dy.double(), uw, out[-2].cpu().double(), out[-1].cpu().double(), wd,
                      dsum.double() if residual else None)
    # a row of one value has du = 0 from terms of the size of rstd
    close(du, ref[0], "du", scale=max(float(ref[0].abs().max()), float(out[-1].abs().max())))
    many = math.sqrt(rows)
    close(dw, ref[1], "dweight", scale=max(float(ref[1].abs().max()), many))
    close(db, ref[2], "dbias", scale=max(float(ref[2].abs().max()), many))


@pytest.mark.parametrize("residual", [False, True], ids=["alone", "residual"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", LN_SIZES)
def test_layernorm_sizes(ops, path, rows, n, dtype, residual):
    check_ln(ops, rows, n, dtype, residual)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(20, 100), (7, 64), (65, 1000), (3, 4099)])
def test_layernorm_backward_from_8_bits(ops, path, rows, n, dtype):
    check_ln(ops, rows, n, dtype, residual=True, act=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [64, 200, 1024])
def test_layernorm_slices_of_wider_tensors(ops, path, n, dtype):
    check_ln(ops, 9, n, dtype, residual=True, wide=True)


@pytest.mark.parametrize("n", [96, 3000])
def test_layernorm_without_weights(ops, path, n):
    check_ln(ops, 10, n, "f32", residual=False, affine=False)


def test_layernorm_many_rows(ops, path):
    """More rows than one sweep of the grid: the column sums come from many parts."""
    check_ln(ops, 20011, 40, "f32", residual=False)
    check_ln(ops, 7001, 264, "bf16", residual=True)


def test_layernorm_constant_rows(ops, path):
    """Variance 0: rstd is 1 / sqrt(eps) and y the bias, whatever the row's level."""
    x = torch.full((4, 96), 1000.0, device="cuda")
    w, b = torch.randn(96, device="cuda"), torch.randn(96, device="cuda")
    y, mean, rstd = ops.layernorm_forward(x, w, b, eps=1e-5)
    assert torch.equal(y, b.expand(4, 96)) and torch.equal(mean, x[:, 0])
    close(rstd, torch.full((4,), 1e-5 ** -0.5, dtype=torch.float64), "rstd")


def test_layernorm_large_offset(ops, path):
    """A mean of 1000 spreads: the variance is taken about the mean, in a second sum."""
    g = torch.Generator().manual_seed(1)
    x = 1000 + torch.randn(6, 512, generator=g)
    y, mean, rstd = ops.layernorm_forward(x.cuda())
    _, rm, rr = ln_forward(x.double(), None, None, 1e-5)
    close(mean, rm, "mean")
    close(rstd, rr, "rstd")
    # x - mean carries the mean's own rounding, half of 2^-14 at 1000
    ref = (x.double() - mean.cpu().double()[:, None]) * rstd.cpu().double()[:, None]
    close(y, ref, "y")


def test_layernorm_non_finite_rows_stay_apart(ops, path):
    x, _, dy, _, w, b = (t.cuda() for t in ln_inputs(8, 200, "f32", 2))
    ok = ops.layernorm_forward(x, w, b)
    x2 = x.clone()
    x2[3, 5], x2[6, 0] = math.nan, math.inf
    got = ops.layernorm_forward(x2, w, b)
    keep = [0, 1, 2, 4, 5, 7]
    assert torch.equal(got[0][keep], ok[0][keep])
    assert bool(torch.isnan(got[0][[3, 6]]).all())


def test_layernorm_leading_dimensions_and_empty(ops):
    x = torch.randn(3, 4, 5, 48, device="cuda")
    y, mean, rstd = ops.layernorm_forward(x)
    assert y.shape == x.shape and mean.shape == (3, 4, 5)
    close(y, ln_forward(x.cpu().double(), None, None, 1e-5)[0], "y")
    part = x[:, :, 1]  # rows that are not evenly spaced
    close(ops.layernorm_forward(part)[0], ln_forward(part.cpu().double(), None, None, 1e-5)[0], "y")
    e = torch.empty(0, 16, device="cuda")
    assert ops.layernorm_forward(e)[0].shape == (0, 16)
    z = torch.empty(0, device="cuda")
    _, dw, db = ops.layernorm_backward(e, e, z, z)
    assert not bool(dw.any()) and not bool(db.any())


def test_layernorm_gradient_against_differences(ops):
    rows, n = 5, 37
    x, _, dy, _, w, b = ln_inputs(rows, n, "f32", 3)
    _, mean, rstd = ops.layernorm_forward(x.cuda(), w.cuda(), b.cuda())
    got = ops.layernorm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    ins = [t.double() for t in (x, w, b)]
    g = torch.Generator().manual_seed(4)

    def loss():
        return float((ln_forward(*ins, 1e-5)[0] * dy.double()).sum())
    for k, grad in enumerate(got):
        flat = ins[k].view(-1)
        for at in torch.randint(0, flat.numel(), (12,), generator=g).tolist():
            keep, step = float(flat[at]), 1e-5
            flat[at] = keep + step
            up = loss()
            flat[at] = keep - step
            down = loss()
            flat[at] = keep
            top = float(grad.abs().max())
            assert abs((up - down) / (2 * step) - float(grad.view(-1)[at])) <= F32 * top + 1e-7


def test_layernorm_is_reproducible(ops, path):
    x, _, dy, _, w, b = (t.cuda() for t in ln_inputs(9000, 96, "bf16", 5))
    _, mean, rstd = ops.layernorm_forward(x, w, b)
    a = ops.layernorm_backward(dy, x, mean, rstd, w)
    for _ in range(3):
        for p, q in zip(a, ops.layernorm_backward(dy, x, mean, rstd, w)):
            assert torch.equal(p, q)


# --------------------------------------------------------------------------- 8-bit checkpoints

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(1, 1), (2, 63), (3, 64), (2, 65), (5, 200), (4, 256), (1, 1000)])
def test_act8_codes(ops, path, rows, n, dtype):
    g = torch.Generator().manual_seed(n)
    x = (torch.randn(rows, n, generator=g) * torch.exp2(torch.randint(-30, 30, (rows, n), generator=g))
         ).to(DT[dtype])
    codes, exps = ops.act8_pack(x.cuda())
    rc, re = act8(x.double())
    assert torch.equal(codes.cpu(), rc) and torch.equal(exps.cpu(), re)
    for out in (torch.float32, torch.bfloat16):
        y = ops.act8_unpack(codes, exps, dtype=out)
        assert torch.equal(y.cpu().double(), act8_values(rc, re))  # 8 significant bits: exact in both


def test_act8_values_at_the_edges(ops, path):
    """Zero blocks, the largest and smallest numbers, ties to even, a largest
    value at exactly 127 steps and just above, NaN and infinities."""
    big, tiny = 3.4028234663852886e38, 1.4e-45
    rows = [[0.0] * 64, [big] + [1.0] * 63, [tiny] * 64, [1.1754943508222875e-38] * 64,
            [127.0, 0.5, 1.5, 2.5, -0.5, -1.5] + [0.0] * 58,
            [127.00001, 0.5, 1.5, 2.5, -0.5, -1.5] + [0.0] * 58,
            [math.nan, math.inf, -math.inf, 3.0] + [0.25] * 60, [math.inf] * 64, [-big] * 64]
    x = torch.tensor(rows)
    codes, exps = ops.act8_pack(x.cuda())
    rc, re = act8(x.double())
    assert torch.equal(codes.cpu(), rc) and torch.equal(exps.cpu(), re)
    y = ops.act8_unpack(codes, exps).cpu().double()
    ref = act8_values(rc, re)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(ref))


def test_act8_slices_and_empty(ops, path):
    big = torch.randn(7, 500, device="cuda")
    part = big[:, 101:301]
    codes, exps = ops.act8_pack(part)
    rc, re = act8(part.cpu().double())
    assert torch.equal(codes.cpu(), rc) and torch.equal(exps.cpu(), re)
    e = torch.empty(0, 70, device="cuda")
    codes, exps = ops.act8_pack(e)
    assert exps.shape == (0, 2) and ops.act8_unpack(codes, exps).shape == (0, 70)


# --------------------------------------------------------------------------- streams, graphs, handle

def test_another_stream(ops):
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(300, 2, 64, "bf16", 14))
    torch.cuda.synchronize()
    want = ops.linrec_forward(x, r, i, lam, h0=h0, states=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.linrec_forward(x, r, i, lam, h0=h0, states=True, stream=side)
    back = ops.linrec_backward(x, x, r, i, lam, got[2], stream=side.cuda_stream)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in zip(back, ops.linrec_backward(x, x, r, i, lam, want[2])):
        assert torch.equal(a, b)


def test_calls_in_a_cuda_graph(ops):
    """Captured once, replayed with other inputs in the same buffers."""
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(700, 2, 128, "bf16", 15))
    w, b = torch.randn(128, device="cuda"), torch.randn(128, device="cuda")

    def passes():
        n, mean, rstd = ops.layernorm_forward(x, w, b)
        y, _, st = ops.linrec_forward(n, r, i, lam, h0=h0, states=True)
        dn, dr, di, dlam, dh0 = ops.linrec_backward(y, *(ops.act8_pack(t) for t in (n, r, i)), lam, st)
        return (y, dr, di, dlam, dh0, *ops.layernorm_backward(dn, x, mean, rstd, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        passes()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = passes()
    for seed in (16, 17):
        for t, v in zip((x, r, i), rec_inputs(700, 2, 128, "bf16", seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for p, q in zip(got, passes()):
            assert torch.equal(p, q)


def test_launches_and_profile(ops):
    x = torch.randn(64, 96, device="cuda")
    ops.set_attr(binding.RCU_ATTR_PROFILE, 1)
    try:
        _, mean, rstd = ops.layernorm_forward(x)
        assert ops.launch_count() == 1
        ops.layernorm_backward(x, x, mean, rstd)
        assert ops.launch_count() >= 1
        p = ops.profile()
        assert p["layernorm_forward"][1] == 1 and p["layernorm_backward"][0] > 0
    finally:
        ops.set_attr(binding.RCU_ATTR_PROFILE, 0)
        binding.load().rcu_seq_profile_reset(ops.h)


# --------------------------------------------------------------------------- refusals

def test_refusals(ops):
    x = torch.randn(4, 2, 8, device="cuda")
    lam, st = torch.zeros(8, device="cuda"), torch.zeros(1, 2, 8, device="cuda")
    bad = [
        lambda: ops.linrec_forward(x.half(), x, x, lam),
        lambda: ops.linrec_forward(x, x.bfloat16(), x, lam),
        lambda: ops.linrec_forward(x, x[:3], x, lam),
        lambda: ops.linrec_forward(x, x, x, lam[:7]),
        lambda: ops.linrec_forward(x, x, x, lam.double()),
        lambda: ops.linrec_forward(x, x, x, lam.cpu()),
        lambda: ops.linrec_forward(x[0], x[0], x[0], lam),
        lambda: ops.linrec_forward(x, x, x, lam, lengths=torch.zeros(2, device="cuda")),
        lambda: ops.linrec_forward(x, x, x, lam, h0=lam),
        lambda: ops.linrec_backward(x, x, x, ops.act8_pack(x), lam, st),
        lambda: ops.linrec_backward(x, x, x, x, lam, st[:0]),
        lambda: ops.linrec_step(x[0], x[0], x[0], lam, torch.zeros(2, 7, device="cuda")),
        lambda: ops.linrec_step(x[0], x[0], x[0], lam, torch.zeros(8, 2, device="cuda").t()),
        lambda: ops.layernorm_forward(x, residual=x[:2]),
        lambda: ops.layernorm_forward(x, weight=lam[:3]),
        lambda: ops.layernorm_backward(x, x, st, st),
        lambda: ops.act8_pack(x.double()),
        lambda: ops.act8_unpack(x, x),
        lambda: ops.act8_unpack(*ops.act8_pack(x), dtype=torch.float16),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {k} was taken")
    for c in (0.0, -1.0, math.nan, math.inf, 1e-60):
        with pytest.raises(binding.RcuError) as e:
            ops.linrec_forward(x, x, x, lam, c=c)
        assert e.value.code == binding.RCU_ERR_INVALID
    with pytest.raises(binding.RcuError):
        ops.layernorm_forward(x, eps=-1.0)
    with pytest.raises(binding.RcuError):
        ops.linrec_step(x[0], x[0], x[0], lam, torch.zeros(1, 8, device="cuda"))
    with pytest.raises(binding.RcuError):
        ops.set_attr(binding.RCU_ATTR_TRACE, 1)
    assert ops.status() == 0


def test_c_entry_refusals(ops):
    """What the wrapper never passes: NULL operands, overlapping rows, bad enums."""
    lib, h = binding.load(), ops.h
    x = torch.randn(4, 2, 8, device="cuda")
    p, lam = x.data_ptr(), torch.zeros(8, device="cuda").data_ptr()

    def fwd(dtype=0, layout=0, T=4, B=2, H=8, x=p, ldx=8, lam=lam, y=p):
        return lib.rcu_linrec_forward(h, dtype, layout, T, B, H, x, ldx, p, 8, p, 8, lam, 8.0, None,
                                      None, y, 8, None, None, None)
    for kw in (dict(dtype=2), dict(dtype=7), dict(layout=2), dict(T=-1), dict(B=-1), dict(H=0),
               dict(x=None), dict(ldx=7), dict(lam=None), dict(y=None)):
        assert fwd(**kw) == binding.RCU_ERR_INVALID, kw

    def bwd(saved=0, e=None, states=p):
        return lib.rcu_linrec_backward(h, 0, saved, 0, 4, 2, 8, p, 8, p, 8, p, 8, e, e, e, lam, 8.0,
                                       None, states, p, 8, None, None, 8, None, 8, None, 8, None,
                                       None, None)
    for kw in (dict(saved=1), dict(saved=2), dict(e=p), dict(states=None)):
        assert bwd(**kw) == binding.RCU_ERR_INVALID, kw

    def ln(n=8, rows=8, ldx=8, res=None, out=None):
        return lib.rcu_layernorm_forward(h, 0, rows, n, p, ldx, res, 8, None, None, 1e-5, p, 8, out,
                                         8, None, None, None)
    for kw in (dict(n=0), dict(rows=-1), dict(ldx=7), dict(res=p), dict(out=p)):
        assert ln(**kw) == binding.RCU_ERR_INVALID, kw
    assert lib.rcu_act8_pack(h, 0, 8, 8, p, 8, p, 8, None, None) == binding.RCU_ERR_INVALID
    assert lib.rcu_act8_unpack(h, 0, 8, 8, None, 8, p, p, 8, None) == binding.RCU_ERR_INVALID
    torch.cuda.synchronize()
    assert ops.status() == 0


# --------------------------------------------------------------------------- together

def test_backward_into_a_fused_gradient(ops, path):
    T, B, H = 130, 2, 72
    x, r, i, lam, h0 = (t.cuda() for t in rec_inputs(T, B, H, "bf16", 18))
    z = torch.cat([x, r, i], -1)
    parts = z.chunk(3, -1)
    y, _, st = ops.linrec_forward(*parts, lam, h0=h0, states=True)
    dy = torch.randn_like(y)
    want = ops.linrec_backward(dy, x, r, i, lam, st)
    dz = torch.full_like(z, 7.0)
    got = ops.linrec_backward(dy, *parts, lam, st, out=dz)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(dz, torch.cat(want[:3], -1))
    with pytest.raises(ValueError):
        ops.linrec_backward(dy, *parts, lam, st, out=dz[..., :-1])


@pytest.mark.parametrize("act8", [False, True])
def test_block_gradients(act8):
    """The stack's gradients against torch autograd on the same formulas in 64
    bits (fp32 products); from 8-bit checkpoints within their steps."""
    from recurrent_cell_unroll_gb300.linrec_block import C, LinRecStack
    net = LinRecStack(2, 24, 40, dtype=torch.float32)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(70, 3, 24, generator=g)
    lengths = torch.tensor([70, 33, 1])
    y, state = net.forward(x.cuda(), lengths=lengths.int().cuda(), act8=act8)
    wy, ws = torch.randn(y.shape, generator=g), torch.randn(state.shape, generator=g)
    ((y * wy.cuda()).sum() + (state * ws.cuda()).sum()).backward()
    leaves = [{k: t.detach().cpu().double().requires_grad_() for k, t in b.items()} for b in net.blocks]
    u, v, after = x.double(), torch.zeros_like(x).double(), []
    for b in leaves:
        u = u + v
        n, _, _ = ln_forward(u, b["weight"], b["bias"], 1e-5)
        out, h, _ = rec_forward(*(n @ b["w_in"]).chunk(3, -1), b["lam"], C, lengths, None)
        v = out @ b["w_out"]
        after.append(h)
    (((u + v) * wy.double()).sum() + (torch.stack(after) * ws.double()).sum()).backward()
    close(y, (u + v).detach(), "y")
    for b, ref in zip(net.blocks, leaves):
        for k, t in b.items():
            top = float(ref[k].grad.abs().max())
            off = float((t.grad.cpu().double() - ref[k].grad).abs().max())
            # products in fp32 (TF32 is off by default) round some 2^-20 of their terms' scale;
            # 8 bits: half a step of 1/63 of a block's largest value, of either sign
            assert off <= (0.05 if act8 else 1e-4) * top, (k, off, top)


@pytest.mark.parametrize("act8", [False, True])
def test_example_trains_and_serves(act8):
    from recurrent_cell_unroll_gb300 import linrec_block
    losses, off = linrec_block.main(["--steps", "40"] + (["--act8"] if act8 else []))
    assert losses[-1] < 0.8 * losses[0]
    assert off <= 2e-2  # two passes of bf16 activations
