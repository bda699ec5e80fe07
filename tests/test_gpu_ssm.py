"""GPU parity of the short causal convolution and the selective scan (forward,
backward, single steps) with plain 64-bit implementations, at the sizes, masks,
strides and values where they can go wrong.

Tolerances: an fp32 result is within F32 of its tensor's largest magnitude.  A
decay is an exponential good to 2^-22 of a rounded argument of at most 2^5 (error
2^-24 * 2^5 / 2), that is about 1e-6, and a sum over the steps that a state
remembers, over states, channels or rows collects at most a few tens of that.  A
bf16 result is rounded once more: half a unit in its last place, 2^-8 of the value.
The gradient of dt is a sum of two terms, through the decays and through the inputs,
that may cancel; each carries that error by itself, so it (and its sum over steps and
rows) is held to F32 of the terms' magnitudes.
"""
import pytest
import torch

import ssm_ref as ref
from recurrent_cell_unroll_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16_HALF = 2e-5, 2.0 ** -8
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


def close(got, want, name, top=None):
    want = want.detach()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if want.numel() == 0:
        return
    half = BF16_HALF if got.dtype == torch.bfloat16 else 0.0
    got = got.detach().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN in other places"
    got, want = torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0)
    top = float(want.abs().max()) if top is None else top
    off = (got - want).abs() - half * want.abs() - F32 * top
    assert float(off.max()) <= 0, f"{name}: off by {float((got - want).abs().max()):.3e} of {top:.3e}"


class Make:
    """Random inputs as the GPU gets them (strided on demand), and in 64 bits as leaves."""

    def __init__(self, seed, dtype, batch_first=False, gap=0):
        self.g = torch.Generator().manual_seed(seed)
        self.dtype, self.batch_first, self.gap = DT[dtype], batch_first, gap

    def __call__(self, *shape, std=1.0, add=0.0, f32=False, rows=False):
        t = torch.randn(shape, generator=self.g) * std + add
        dtype = torch.float32 if f32 else self.dtype
        t = t.to(dtype)
        wide = t.double().requires_grad_()
        if rows and self.batch_first:
            t = t.transpose(0, 1).contiguous()
        if rows and self.gap:  # a slice of a wider tensor
            room = torch.full((*t.shape[:-1], t.shape[-1] + self.gap), float("nan"), dtype=dtype, device="cuda")
            room[..., self.gap:] = t.cuda()
            return room[..., self.gap:], wide
        return t.cuda(), wide

    def back(self, t):
        return t.transpose(0, 1) if self.batch_first else t


def masked(t, lengths, make, value):
    """The GPU's tensor with `value` in every step past its row's end."""
    if lengths is not None:
        view = make.back(t)
        for b, n in enumerate(lengths):
            view[n:, b] = value
    return t


def check_conv(ops, T, B, H, W, dtype, lengths=None, batch_first=False, gap=0, silu=True, bias=True, state=True,
               seed=0):
    make = Make(seed + T, dtype, batch_first, gap)
    x, rx = make(T, B, H, rows=True)
    w, rw = make(H, W, std=0.5, f32=True)
    bi, rb = make(H, std=0.5, f32=True) if bias else (None, None)
    st, rs = make(B, W - 1, H) if state else (None, None)
    dy, rdy = make(T, B, H, rows=True)
    ds, rds = make(B, W - 1, H)
    masked(x, lengths, make, float("inf"))
    masked(dy, lengths, make, float("nan"))
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
    how = {"bias": bi, "silu": silu, "lengths": ln, "state": st, "batch_first": batch_first}
    y, end = ops.conv_forward(x, w, **how)
    want, wend = ref.conv(rx, rw, rb, silu, lengths, rs)
    close(make.back(y), want, "y")
    close(end, wend, "state_n")
    leaves = [t for t in (rx, rw, rb, rs) if t is not None]
    grads = dict(zip(map(id, leaves), torch.autograd.grad((want, wend), leaves, (rdy, rds), allow_unused=True)))

    def grad(t):
        g = grads[id(t)]
        return torch.zeros_like(t) if g is None else g
    dx, dw, db, dst = ops.conv_backward(dy, x, w, dstate_n=ds, **how)
    close(make.back(dx), grad(rx), "dx")
    close(dw, grad(rw), "dweight")
    if bias:
        close(db, grad(rb), "dbias")
    if state:
        close(dst, grad(rs), "dstate")
    assert ops.status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,W,kw", [
    (1, 1, 1, 1, {}), (1, 2, 8, 4, {}), (2, 3, 16, 4, {}), (3, 1, 24, 8, {}), (40, 3, 40, 4, {}),
    (70, 2, 33, 3, {"gap": 5}), (130, 2, 64, 2, {"gap": 8, "batch_first": True}), (200, 1, 8, 4, {"silu": False}),
    (33, 2, 20, 5, {"bias": False}), (64, 5, 48, 4, {"state": False, "batch_first": True}),
    (50, 6, 16, 4, {"lengths": [0, 1, 2, 3, 50, 49]}), (50, 4, 9, 8, {"lengths": [0, 5, 6, 50]}),
    (300, 3, 16, 3, {"lengths": [17, 0, 300], "state": False}), (1, 700, 64, 4, {}), (20, 3, 1000, 4, {})])
def test_conv(ops, path, dtype, T, B, H, W, kw):
    check_conv(ops, T, B, H, W, dtype, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,W,kw", [
    (50, 6, 10, 4, {"lengths": [0, 1, 2, 3, 50, 49]}), (50, 6, 11, 3, {"lengths": [0, 1, 2, 3, 50, 49]}),
    (70, 7, 22, 6, {"lengths": [0, 1, 4, 5, 6, 70, 64]}), (70, 4, 21, 7, {"lengths": [3, 70, 0, 69], "gap": 2}),
    (41, 3, 6, 1, {"lengths": [41, 0, 7]}), (2, 900, 1001, 4, {}), (1, 700, 1002, 8, {}), (301, 2, 34, 5, {"gap": 2}),
    (9, 2, 1, 4, {}), (9, 2, 2, 8, {"batch_first": True})])
def test_conv_in_pairs(ops, dtype, T, B, H, W, kw):
    """Widths of two, not of four channels, odd ones, and unusual numbers of taps."""
    check_conv(ops, T, B, H, W, dtype, **kw)


def test_conv_rows_beyond_the_gpu(ops):
    """More rows than threads: a thread takes several, and their sums."""
    check_conv(ops, 3, 3000, 1024, 4, "bf16", lengths=[b % 4 for b in range(3000)])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [1, 2, 4, 7])
def test_conv_steps_follow_the_sequence(ops, path, dtype, W):
    """A prompt, then steps with slots: as one sequence; rows without a slot stay out."""
    T, B, H, slots = 9, 5, 20, 11
    make = Make(W, dtype)
    x, _ = make(T, B, H)
    w, _ = make(H, W, std=0.5, f32=True)
    bias, _ = make(H, f32=True)
    whole, end = ops.conv_forward(x, w, bias=bias)
    _, table = ops.conv_forward(x[:5], w, bias=bias)
    slot = torch.tensor([10, 3, 7, 0, 4], dtype=torch.int32).cuda()
    room = torch.full((slots, W - 1, H), 7.0, dtype=DT[dtype], device="cuda")
    room[slot.long()] = table
    for t in range(5, T):
        y = ops.conv_step(x[t], w, room, bias=bias, slot=slot)
        assert torch.equal(y, whole[t])
    assert torch.equal(room[slot.long()], end)
    rest = [s for s in range(slots) if s not in slot.tolist()]
    before = room.clone()
    assert bool((room[rest] == 7).all())
    out = torch.full_like(slot, -1)
    out[1] = 3
    y = ops.conv_step(x[0], w, room, bias=bias, slot=out)
    assert bool((y[[0, 2, 3, 4]] == 0).all())
    before[3] = room[3]
    assert torch.equal(room, before) and ops.status() == 0


def scan_inputs(make, T, B, H, N, d=True, bias=True, gate=True, h0=True):
    x, rx = make(T, B, H, rows=True)
    dt, rdt = make(T, B, H, add=0.0 if bias else -3.0, rows=True)
    al, ral = make(H, N, std=0.7, add=0.5, f32=True)
    b, rb = make(T, B, N, rows=True)
    c, rc = make(T, B, N, rows=True)
    dd, rd = make(H, f32=True) if d else (None, None)
    db, rdb = make(H, add=-3.0, f32=True) if bias else (None, None)
    z, rz = make(T, B, H, rows=True) if gate else (None, None)
    h, rh = make(B, H, N, f32=True) if h0 else (None, None)
    return (x, dt, al, b, c, dd, db, z, h), (rx, rdt, ral, rb, rc, rd, rdb, rz, rh)


def check_scan(ops, T, B, H, N, dtype, lengths=None, batch_first=False, gap=0, seed=0, **parts):
    make = Make(seed + T + N, dtype, batch_first, gap)
    (x, dt, al, b, c, d, db, z, h), leaves = scan_inputs(make, T, B, H, N, **parts)
    for t, bad in ((x, float("nan")), (dt, float("inf")), (b, float("nan")), (c, float("inf"))):
        masked(t, lengths, make, bad)
    if z is not None:
        masked(z, lengths, make, float("nan"))
    ln = torch.tensor(lengths, dtype=torch.int32) if lengths is not None else None
    how = {"d": d, "dt_bias": db, "z": z, "lengths": ln.cuda() if ln is not None else None,
           "batch_first": batch_first}
    y, h_n, states = ops.selscan_forward(x, dt, al, b, c, h0=h, states=True, **how)
    want, wh, wstates = ref.scan(*leaves[:8], ln, leaves[8])
    close(make.back(y), want, "y")
    close(h_n, wh, "h_n")
    close(states, wstates, "states")
    again = ops.selscan_forward(x, dt, al, b, c, h0=h, **how)
    assert torch.equal(again[0], y) and torch.equal(again[1], h_n) and again[2] is None
    dy, rdy = make(T, B, H, rows=True)
    masked(dy, lengths, make, float("nan"))
    dh, rdh = make(B, H, N, f32=True)
    there = [t for t in leaves if t is not None]
    grads = dict(zip(map(id, there), torch.autograd.grad((want, wh), there, (rdy, rdh))))
    got = ops.selscan_backward(dy, x, dt, al, b, c, states, dh_n=dh, **how)
    names = ("dx", "ddt", "da_log", "db", "dc", "dd", "ddt_bias", "dz", "dh0")
    apart = leaves[1].detach().requires_grad_()
    split = ref.scan(*leaves[:8], ln, leaves[8], dt_in=apart)[:2]
    terms = sum(t.abs() for t in torch.autograd.grad(split, (leaves[1], apart), (rdy, rdh)))
    tops = {"ddt": float(terms.max()), "ddt_bias": float(terms.sum((0, 1)).max())}
    for name, leaf in zip(names, leaves):
        if leaf is None:
            assert name == "dh0" or got[name] is None
            continue
        g = got[name]
        close(make.back(g) if name in ("dx", "ddt", "db", "dc", "dz") else g, grads[id(leaf)], name,
              tops.get(name))
    twice = ops.selscan_backward(dy, x, dt, al, b, c, states, dh_n=dh, **how)
    for name in names:  # sums in a fixed order
        assert got[name] is None or torch.equal(got[name], twice[name]), name
    assert ops.status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,N,kw", [
    (1, 1, 1, 1, {}), (1, 2, 64, 16, {}), (2, 1, 8, 8, {}), (5, 3, 33, 5, {}), (31, 2, 20, 16, {}),
    (32, 1, 128, 16, {"gate": False}), (33, 2, 130, 16, {"d": False}), (64, 1, 64, 16, {"bias": False}),
    (67, 2, 70, 16, {"gap": 3}), (100, 2, 136, 16, {"gap": 8, "batch_first": True, "h0": False}),
    (40, 2, 24, 64, {}), (45, 1, 50, 33, {}), (70, 2, 40, 24, {}), (35, 1, 65, 7, {"gap": 1}), (64, 3, 40, 32, {}),
    (70, 5, 40, 16, {"lengths": [0, 1, 70, 32, 33]}), (97, 4, 24, 3, {"lengths": [64, 0, 97, 96], "gap": 2}),
    (97, 3, 24, 40, {"lengths": [65, 0, 31], "batch_first": True}),
    (700, 1, 64, 16, {}), (515, 2, 72, 8, {"lengths": [515, 140]}), (400, 2, 16, 64, {"lengths": [31, 400]})])
def test_scan(ops, path, dtype, T, B, H, N, kw):
    check_scan(ops, T, B, H, N, dtype, **kw)


def test_scan_long(ops):
    """Many segments, chained."""
    check_scan(ops, 6000, 1, 8, 16, "f32")
    check_scan(ops, 5003, 2, 10, 5, "bf16", lengths=[3000, 5003])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 4, 6, 8, 16, 30, 32, 64])
def test_scan_steps_follow_the_sequence(ops, path, dtype, N):
    T, B, H, slots = 12, 5, 37, 9
    make = Make(N, dtype)
    (x, dt, al, b, c, d, db, z, h0), leaves = scan_inputs(make, T, B, H, N)
    want, wh, _ = ref.scan(*leaves[:8], None, leaves[8])
    slot = torch.tensor([8, 3, 7, 0, 4], dtype=torch.int32).cuda()
    room = torch.full((slots, H, N), 7.0, device="cuda")
    room[slot.long()] = ops.selscan_forward(*(t[:5] for t in (x, dt)), al, *(t[:5] for t in (b, c)), d=d, dt_bias=db,
                                            z=z[:5], h0=h0)[1]
    for t in range(5, T):
        y = ops.selscan_step(x[t], dt[t], al, b[t], c[t], room, d=d, dt_bias=db, z=z[t], slot=slot)
        close(y, want[t], f"y at {t}")
    close(room[slot.long()], wh, "states")
    rest = [s for s in range(slots) if s not in slot.tolist()]
    assert bool((room[rest] == 7).all())
    out = torch.full_like(slot, -1)
    out[1] = 3
    before = room.clone()
    y = ops.selscan_step(x[0], dt[0], al, b[0], c[0], room, d=d, dt_bias=db, z=z[0], slot=out)
    assert bool((y[[0, 2, 3, 4]] == 0).all())
    before[3] = room[3]
    assert torch.equal(room, before)
    # without slots, gate and skip; rows b of the table
    room = torch.zeros(B, H, N, device="cuda")
    y = ops.selscan_step(x[0], dt[0], al, b[0], c[0], room)
    w, wh, _ = ref.scan(*(t[:1] for t in leaves[:2]), leaves[2], *(t[:1] for t in leaves[3:5]), None, None, None,
                        None, None)
    close(y, w[0], "y")
    close(room, wh, "states")
    assert ops.status() == 0


def test_scan_gradients_against_differences(ops):
    """Central differences of the kernels' own forward, in directions at random."""
    T, B, H, N = 21, 2, 10, 6
    make = Make(5, "f32")
    args, _ = scan_inputs(make, T, B, H, N)
    names = ("x", "dt", "a_log", "b", "c", "d", "dt_bias", "z", "h0")
    at = dict(zip(names, args))
    dy, _ = make(T, B, H)
    dh, _ = make(B, H, N, f32=True)

    def loss(v):
        y, h, _ = ops.selscan_forward(**v)
        return float((y.double() * dy).sum() + (h.double() * dh).sum())
    states = ops.selscan_forward(**at, states=True)[2]
    got = ops.selscan_backward(dy, **{k: v for k, v in at.items() if k != "h0"}, states=states, dh_n=dh)
    for name in names:
        way = torch.randn(at[name].shape, generator=make.g).cuda()
        eps = 1e-3
        up, down = (loss({**at, name: at[name] + s * eps * way}) for s in (1, -1))
        slope = (up - down) / (2 * eps)
        mine = float((got["da_log" if name == "a_log" else "d" + name].double() * way).sum())
        # rounding: values of some 100 in all, kept to 1e-6 of that, over 2 eps; curvature: eps^2
        assert abs(slope - mine) <= 0.1 + 2e-3 * abs(mine), (name, slope, mine)


def test_conv_gradients_against_differences(ops):
    make = Make(6, "f32")
    T, B, H, W = 13, 2, 6, 4
    at = {"x": make(T, B, H)[0], "weight": make(H, W)[0], "bias": make(H)[0], "state": make(B, W - 1, H)[0]}
    dy, ds = make(T, B, H)[0], make(B, W - 1, H)[0]

    def loss(v):
        y, s = ops.conv_forward(**v)
        return float((y.double() * dy).sum() + (s.double() * ds).sum())
    got = ops.conv_backward(dy, **at, dstate_n=ds)
    for name, g in zip(("x", "weight", "bias", "state"), got):
        way = torch.randn(at[name].shape, generator=make.g).cuda()
        up, down = (loss({**at, name: at[name] + s * 1e-3 * way}) for s in (1, -1))
        mine = float((g.double() * way).sum())
        assert abs((up - down) / 2e-3 - mine) <= 0.05 + 2e-3 * abs(mine), (name, mine)


def test_infinite_and_nan_inputs(ops):
    """As the formulas have them: a step of -inf changes nothing, one of a large logit
    forgets, a NaN stays in its channel and its row."""
    T, B, H, N = 40, 2, 40, 16
    make = Make(3, "f32")
    (x, dt, al, b, c, d, db, z, h0), leaves = scan_inputs(make, T, B, H, N)
    cases = [(0, 1, 5, -float("inf")), (7, 0, 3, 80.0), (20, 1, 9, float("nan")), (12, 0, 30, -200.0)]
    leaves = [t.detach() for t in leaves]
    for t, row, ch, v in cases:
        dt[t, row, ch] = v
        leaves[1][t, row, ch] = v
    al[4, 2] = leaves[2][4, 2] = float("-inf")  # a state that does not decay
    al[6, 1] = leaves[2][6, 1] = 200.0          # one that forgets at once: exp(a_log) is infinite in fp32
    y, h, _ = ops.selscan_forward(x, dt, al, b, c, d=d, dt_bias=db, z=z, h0=h0)
    want, wh, _ = ref.scan(*leaves[:8], None, leaves[8])
    close(y, want, "y")
    close(h, wh, "h_n")
    assert int(torch.isnan(y).sum()) == T - 20


def test_large_strides_pass_32_bits(ops):
    """Rows further apart than 2^31 elements."""
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    H, far = 64, (1 << 31) + 64
    room = torch.zeros(2 * far, dtype=torch.bfloat16, device="cuda")
    x = room.as_strided((2, 3, H), (far, H, 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randn(2, 3, H, generator=g, device="cuda").bfloat16()
    x.copy_(v)
    w = torch.randn(H, 4, generator=g, device="cuda")
    big = room.as_strided((2, 3, H), (far, far // 4, 1))
    big.copy_(v)
    wide = big.transpose(0, 1)  # rows of one batch entry far apart: batch first [3, 2, H]
    y, _ = ops.conv_forward(v.transpose(0, 1).contiguous(), w, batch_first=True)
    assert torch.equal(y, ops.conv_forward(wide, w, batch_first=True)[0])
    al = torch.zeros(H, 4, device="cuda")
    b = torch.randn(2, 3, 4, generator=g, device="cuda").bfloat16()
    one = room.as_strided((6, 1, H), (far // 4, far // 4, 1))  # evenly spaced rows, in place
    one.copy_(v.reshape(6, 1, H))
    args = (al, b.reshape(6, 1, 4), b.reshape(6, 1, 4))
    want = ops.selscan_forward(v.reshape(6, 1, H), v.reshape(6, 1, H), *args, states=True)
    got = ops.selscan_forward(one, one, *args, states=True)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    first = ops.selscan_backward(v.reshape(6, 1, H), v.reshape(6, 1, H), v.reshape(6, 1, H), *args, want[2])
    second = ops.selscan_backward(one, one, one, *args, want[2])
    for k, t in first.items():
        assert t is None or torch.equal(t, second[k]), k
    assert ops.status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,W,N,start,gap", [
    (37, 2, 65, 4, 16, 1, 0), (40, 3, 64, 3, 16, 1, 2), (33, 2, 128, 4, 5, 3, 1), (35, 2, 127, 2, 3, 0, 3),
    (18, 1, 1, 4, 1, 1, 2), (20, 2, 63, 5, 33, 1, 0), (45, 2, 66, 8, 32, 2, 0), (300, 2, 61, 4, 16, 1, 5)])
def test_rows_anywhere(ops, dtype, T, B, H, W, N, start, gap):
    """Rows that start and end in the middle of a word, in the midst of NaN: what rows of
    their own give, bit for bit where the rows of both are read one way."""
    make = Make(11, dtype)
    room = {}

    def rows(t):
        wide = t.shape[-1] + gap
        flat = torch.full((start + T * B * wide - gap,), float("nan"), dtype=t.dtype, device="cuda")
        v = flat.as_strided(t.shape, (B * wide, wide, 1), start)
        v.copy_(t)
        room[v.data_ptr()] = flat
        return v

    def around(v):  # the NaN that are left of it
        return int(torch.isnan(room[v.data_ptr()]).sum())

    (x, dt, al, b, c, d, db, z, h0), _ = scan_inputs(make, T, B, H, N)
    w, _ = make(H, W, std=0.5, f32=True)
    dy, _ = make(T, B, H, rows=True)
    x, dt, b, c, z, dy = (t.contiguous() for t in (x, dt, b, c, z, dy))
    px, pdt, pb, pc, pz, pdy = (rows(t) for t in (x, dt, b, c, z, dy))
    how = {"d": d, "dt_bias": db, "h0": h0, "states": True}
    want = ops.selscan_forward(x, dt, al, b, c, z=z, **how)
    got = ops.selscan_forward(px, pdt, al, pb, pc, z=pz, **how)
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    how = {"d": d, "dt_bias": db}
    want = ops.selscan_backward(dy, x, dt, al, b, c, want[2], z=z, **how)
    got = ops.selscan_backward(pdy, px, pdt, al, pb, pc, got[2], z=pz, **how)
    for k, t in want.items():
        assert t is None or torch.equal(t, got[k]), k
    want, got = ops.conv_forward(x, w, bias=d), ops.conv_forward(px, w, bias=d)
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    want, got = ops.conv_backward(dy, x, w, bias=d), ops.conv_backward(pdy, px, w, bias=d)
    assert torch.equal(want[0], got[0])
    # sums over the T B steps, in another order where other words are read: off by at most
    # T B half steps of the sum of their terms' magnitudes, each; silu' is below 1.1
    top = 1.1 * float(dy.abs().sum((0, 1)).max()) * max(float(x.abs().max()), 1.0)
    for p, q in zip(want[1:3], got[1:3]):
        assert (p is None) == (q is None)
        if p is not None:
            assert float((p - q).abs().max()) <= 2 * T * B * 2.0 ** -24 * top
    for v in (px, pdt, pb, pc, pz, pdy):
        assert around(v) == start + (T * B - 1) * gap
    assert ops.status() == 0


def test_lengths_and_slots_out_of_range_are_reported(ops):
    make = Make(1, "f32")
    (x, dt, al, b, c, *_), _ = scan_inputs(make, 8, 3, 10, 4)
    bad = torch.tensor([-1, 9, 3], dtype=torch.int32).cuda()
    good = torch.tensor([0, 8, 3], dtype=torch.int32).cuda()
    w = torch.randn(10, 4, device="cuda")
    for call in (lambda n: ops.conv_forward(x, w, lengths=n)[0],
                 lambda n: ops.conv_backward(x, x, w, lengths=n)[0],
                 lambda n: ops.selscan_forward(x, dt, al, b, c, lengths=n)[0],
                 lambda n: ops.selscan_backward(x, x, dt, al, b, c, torch.zeros(1, 3, 10, 4, device="cuda"),
                                                lengths=n)["dx"]):
        got = call(bad)
        assert ops.status() == binding.RCU_ERR_LENGTHS
        assert torch.equal(got, call(good)) and ops.status() == 0
    slot = torch.tensor([0, 3, -2], dtype=torch.int32).cuda()
    window, states = torch.zeros(3, 3, 10, device="cuda"), torch.zeros(3, 10, 4, device="cuda")
    y = ops.conv_step(x[0], w, window, slot=slot)
    assert ops.status() == binding.RCU_ERR_SLOTS and bool((y[1:] == 0).all()) and bool((window[1:] == 0).all())
    y = ops.selscan_step(x[0], dt[0], al, b[0], c[0], states, slot=slot)
    assert ops.status() == binding.RCU_ERR_SLOTS and bool((y[1:] == 0).all()) and bool((states[1:] == 0).all())


def test_empty(ops):
    al, w = torch.zeros(4, 3, device="cuda"), torch.zeros(4, 3, device="cuda")
    for T, B in ((0, 2), (3, 0), (0, 0)):
        x, b = torch.zeros(T, B, 4, device="cuda"), torch.zeros(T, B, 3, device="cuda")
        h0, st = torch.randn(B, 4, 3, device="cuda"), torch.randn(B, 2, 4, device="cuda")
        y, end = ops.conv_forward(x, w, state=st)
        assert y.shape == x.shape and torch.equal(end, st)
        dx, dw, db, ds = ops.conv_backward(x, x, w, state=st, dstate_n=st)
        assert not dw.any() and not db.any() and torch.equal(ds, st)
        y, h, states = ops.selscan_forward(x, x, al, b, b, h0=h0, states=True)
        assert torch.equal(h, h0)
        g = ops.selscan_backward(x, x, x, al, b, b, states, dh_n=h0)
        assert torch.equal(g["dh0"], h0) and not g["da_log"].any()
    assert ops.conv_step(torch.zeros(0, 4, device="cuda"), w, torch.zeros(2, 2, 4, device="cuda")).shape == (0, 4)
    assert ops.status() == 0


def test_state_in_place(ops):
    """state_n may be the state itself (the C call): a prompt in pieces."""
    import ctypes
    g = torch.Generator(device="cuda").manual_seed(2)
    for T in (1, 2, 9):
        x = torch.randn(T, 3, 16, generator=g, device="cuda")
        w = torch.randn(16, 4, generator=g, device="cuda")
        st = torch.randn(3, 3, 16, generator=g, device="cuda")
        y, end = ops.conv_forward(x, w, state=st)
        y2 = torch.empty_like(y)
        rc = ops.lib.rcu_conv_forward(ops.h, 0, 0, T, 3, 16, 4, x.data_ptr(), 16, w.data_ptr(), None, 1, None,
                                      st.data_ptr(), y2.data_ptr(), 16, st.data_ptr(), ctypes.c_void_p(
                                          torch.cuda.current_stream().cuda_stream))
        assert rc == 0 and torch.equal(y, y2) and torch.equal(end, st)


def test_captured_and_on_another_stream(ops):
    make = Make(9, "bf16")
    T, B, H, N = 600, 2, 24, 16
    (x, dt, al, b, c, d, db, z, h0), _ = scan_inputs(make, T, B, H, N)
    w = torch.randn(H, 4, device="cuda")
    dy = torch.randn(T, B, H, device="cuda").bfloat16()

    def whole():
        u, end = ops.conv_forward(x, w)
        y, h, st = ops.selscan_forward(u, dt, al, b, c, d=d, dt_bias=db, z=z, h0=h0, states=True)
        g = ops.selscan_backward(dy, u, dt, al, b, c, st, d=d, dt_bias=db, z=z)
        return (y, h, end, *(g[k] for k in sorted(g)), *ops.conv_backward(g["dx"], x, w))
    want = [t.clone() for t in whole()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = ops.selscan_forward(x, dt, al, b, c, d=d, dt_bias=db, z=z, h0=h0, stream=side)[0]
    side.synchronize()
    assert torch.equal(on_side, ops.selscan_forward(x, dt, al, b, c, d=d, dt_bias=db, z=z, h0=h0)[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = whole()
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b_ in zip(want, out):
        assert torch.equal(a, b_)
    x.mul_(0.5)
    graph.replay()
    for a, b_ in zip(whole(), out):
        assert torch.equal(a, b_)
    assert ops.status() == 0
