"""GPU parity of the AdamW step over lists of tensors (states in 32 and in 8 bits)
with plain 64-bit implementations.

Tolerances.  fp32 states: two products and a sum, each rounded to half a unit: within
2^-22 of the larger of the two terms, taken as 3e-7 of the tensor's largest one.  A
parameter: the update lr m / (sqrt(v) + eps) carries a few roundings of 2^-24 and a
division good to 2 units, below 1e-6 of it, and is added with one rounding of p.
8-bit states round to one of the two codes around the exact value, a step apart.
"""
import math

import pytest
import torch

import ssm_ref as ref
from recurrent_cell_unroll_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


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


SHAPES = [(1,), (7,), (64,), (65, 3), (0,), (2048,), (2049,), (100, 100), (3, 5, 7), (5000,)]


def make(shapes, p_type=F32, g_type=F32, shift=0, seed=0):
    """params, grads, m, v; `shift` values off the start of their buffers."""
    g = torch.Generator().manual_seed(seed)

    def one(shape, dtype, f=lambda t: t):
        n = math.prod(shape)
        room = torch.empty(n + shift, dtype=dtype, device="cuda")
        room[shift:] = f(torch.randn(n, generator=g)).to(dtype).cuda()
        return room[shift:].view(shape)
    return ([one(s, p_type) for s in shapes], [one(s, g_type) for s in shapes], [one(s, F32) for s in shapes],
            [one(s, F32, lambda t: t * t) for s in shapes])


def check_p(got, want, update):
    half = {F32: 2.0 ** -24, BF16: 2.0 ** -8}[got.dtype]
    off = (got.cpu().double() - want).abs() - half * want.abs() * 1.01 - 1e-6 * update.abs() - 1e-7 * want.abs()
    assert off.numel() == 0 or float(off.max()) <= 0, float(off.max())


@pytest.mark.parametrize("p_type,g_type,shift", [(F32, F32, 0), (F32, BF16, 0), (BF16, BF16, 0), (BF16, F32, 0),
                                                 (F32, F32, 1), (BF16, BF16, 3)])
@pytest.mark.parametrize("scaled", [False, True])
def test_states_in_32_bits(ops, path, p_type, g_type, shift, scaled):
    p, g, m, v = make(SHAPES, p_type, g_type, shift)
    how = {"lr": 3e-3, "betas": (0.9, 0.99), "eps": 1e-7, "weight_decay": 0.1}
    scale = torch.tensor([0.37], device="cuda") if scaled else None
    copies = [torch.full(t.shape, 9.0, dtype=BF16, device="cuda") for t in p] if p_type is F32 else None
    want = [ref.adamw(*(t.cpu().double() for t in ts), 5, scale=float(scale) if scaled else None, **how)
            for ts in zip(p, g, m, v)]
    before = [t.cpu().double() for t in p]
    ops.adamw_step(p, g, m, v, 5, scale=scale, copies=copies, **how)
    for k, (wp, wm, wv) in enumerate(want):
        check_p(p[k], wp, wp - before[k])
        if copies is not None:
            assert torch.equal(copies[k], p[k].bfloat16())
        for got, w in ((m[k], wm), (v[k], wv)):
            if w.numel():
                top = max(float(w.abs().max()), float(g[k].double().abs().max() ** 2), 1.0)
                assert float((got.cpu().double() - w).abs().max()) <= 3e-7 * top
    assert ops.status() == 0


def exponent(t):
    top = float(t[torch.isfinite(t)].abs().max()) if torch.isfinite(t).any() else 0.0
    return max(-126, min(126, math.frexp(top)[1] - 1)) if top else -126


def neighbours(value, e, signed):
    """The codes around a value, and where it lies between them."""
    f = abs(value) * 2.0 ** -e
    o = 14 if signed else 30
    lo = 0
    while lo < (127 if signed else 254) - 0 and ref.state8_value((lo + 1) if signed else lo + 1 - 128, 0, signed) <= f:
        lo += 1
    return lo, f, o


@pytest.mark.parametrize("signed", [True, False])
def test_pack_and_unpack(ops, path, signed):
    g = torch.Generator().manual_seed(3)
    for n in (0, 1, 63, 64, 65, 1000, 2049):
        x = torch.randn(n, generator=g) * torch.exp(4 * torch.randn(n, generator=g))
        if not signed:
            x = x * x
        if n > 300:
            x[100:164] = 0
            x[256], x[257] = float("nan"), float("inf")
        codes, exps = ops.state8_pack(x.cuda(), signed)
        got = ops.state8_unpack(codes, exps, signed).cpu().double()
        for k in range(-(-n // 64)):
            part = x[64 * k:64 * k + 64].double()
            e = exponent(part)
            assert int(exps[k]) == e
            for j, value in enumerate(part.tolist()):
                q = int(codes[64 * k + j])
                out = float(got[64 * k + j])
                if not math.isfinite(value):
                    assert q == (-128 if signed else 127) and math.isnan(out)
                    continue
                exact = ref.state8_value(q, e, signed)
                assert abs(out - exact) <= 1e-7 * abs(exact)
                lo, f, _ = neighbours(value, e, signed)
                n_q = abs(q) if signed else q + 128
                assert (q < 0) == (value < 0) or not signed or q == 0
                a, b = (ref.state8_value(i if signed else i - 128, 0, signed) for i in (lo, lo + 1))
                near = lo + (f - a >= (b - a) / 2 * (1 - 1e-6)), lo + (f - a >= (b - a) / 2 * (1 + 1e-6))
                if not signed and value > 0:
                    near = tuple(max(i, 1) for i in near)
                assert n_q in near, (value, e, n_q, near)
        # packing what was unpacked changes nothing
        if n and not torch.isnan(got).any():
            c2, e2 = ops.state8_pack(got.float().cuda(), signed)
            assert torch.equal(ops.state8_unpack(c2, e2, signed).cpu().double(), got)


def step8(ops, p, g, m, v, step, how, seed, place, count):
    """What the kernel should hold: exact codes by the documented hash, from fp32 sums."""
    b1, b2 = (torch.tensor(x, dtype=F32) for x in how["betas"])
    c1, c2 = (torch.tensor(1 - x, dtype=F32) for x in how["betas"])
    m = m * b1 + g * c1
    v = v * b2 + (g * c2) * g
    key = ref.mix((ref.mix((seed + 0x9e3779b9 * step) & 0xffffffff) + place) & 0xffffffff)
    out = []
    for t, signed in ((m, True), (v, False)):
        o = 14 if signed else 30
        codes, exps = [], []
        flat = t.flatten()
        for k in range(0, flat.numel(), 64):
            part = flat[k:k + 64]
            e = exponent(part.double())
            exps.append(e)
            for j, value in enumerate(part):
                if not math.isfinite(float(value)):
                    codes.append(-128 if signed else 127)
                    continue
                word = ref.mix((k + j) ^ key)
                bits = (word & 0xffff if signed else word >> 16) << 4 | 8
                f = (value.abs() * torch.tensor(2.0 ** -e, dtype=F32) + torch.tensor(2.0 ** -o, dtype=F32))
                q = (int(f.view(torch.int32)) + bits >> 20) - ((127 - o) << 3)
                if signed:
                    q = min(q, 127) * (-1 if float(value) < 0 else 1)
                else:
                    q = (max(1, min(q, 254)) if float(value) > 0 else 0) - 128
                codes.append(q)
        out.append((torch.tensor(codes, dtype=torch.int8).view(t.shape), torch.tensor(exps, dtype=torch.int8)))
    return m, v, out


@pytest.mark.parametrize("g_type,shift", [(F32, 0), (BF16, 0), (F32, 1)])
def test_states_in_8_bits(ops, path, g_type, shift):
    """Bit for bit by the documented rounding, over three steps."""
    shapes = [(1,), (64,), (65, 3), (0,), (7,), (2049,)]
    p, g, m, v = make(shapes, F32, g_type, shift, seed=4)
    g[2][0, 1], g[2][3, 2] = float("nan"), float("inf")
    how = {"lr": 1e-2, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.01}

    def odd(t):  # codes that are not aligned either
        room = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        room[shift:] = t.flatten()
        return room[shift:].view(t.shape)
    m8 = [tuple(odd(q) for q in ops.state8_pack(t, True)) for t in m]
    v8 = [tuple(odd(q) for q in ops.state8_pack(t, False)) for t in v]
    for step in (1, 2, 3):
        old = [t.cpu().double() for t in p]
        held = [(ops.state8_unpack(*a, True).cpu(), ops.state8_unpack(*b, False).cpu()) for a, b in zip(m8, v8)]
        ops.adamw_step(p, g, m8, v8, step, seed=11, **how)
        for k, s in enumerate(shapes):
            if math.prod(s) == 0:
                continue
            gm = g[k].float().cpu()
            m1, v1, ((mc, me), (vc, ve)) = step8(ops, p[k], gm, *held[k], step, how, 11, k, len(shapes))
            assert torch.equal(m8[k][0].cpu(), mc) and torch.equal(m8[k][1].cpu(), me), (step, k)
            assert torch.equal(v8[k][0].cpu(), vc) and torch.equal(v8[k][1].cpu(), ve), (step, k)
            wp = ref.adamw(old[k], gm.double(), *(t.double() for t in held[k]), step, how["lr"], how["betas"],
                           how["eps"], how["weight_decay"], None)[0]
            fine = torch.isfinite(wp)
            assert torch.equal(torch.isfinite(p[k].cpu()), fine)
            check_p(p[k][fine.cuda()], wp[fine], (wp - old[k])[fine])
    assert ops.status() == 0


def test_rounding_is_fair(ops):
    """A state that changes by less than a code's step drifts as it should: after 400
    steps with a gradient of 0, v has decayed by beta2^400 on average.

    A step multiplies v by 0.999 and rounds it to one of two codes at most an eighth
    apart, fairly: the mean over n values wanders by at most 1/8 sqrt(400 / n) of them,
    4e-3 here; twelve times that is allowed."""
    n = 1 << 18
    v = torch.rand(n, device="cuda") + 0.5
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m8, v8 = ops.state8_pack(torch.zeros_like(v), True), ops.state8_pack(v, False)
    start = float(ops.state8_unpack(*v8, False).mean())
    for step in range(1, 401):
        ops.adamw_step([p], [g], [m8], [v8], step, betas=(0.9, 0.999), seed=5)
    end = float(ops.state8_unpack(*v8, False).mean())
    assert abs(end / start / 0.999 ** 400 - 1) <= 0.05


def test_many_tensors(ops):
    """More than a launch's table holds; every tensor its own."""
    count = 900
    p, g, m, v = make([(1 + k % 70,) for k in range(count)], seed=7)
    want = [ref.adamw(*(t.cpu().double() for t in ts), 3, 1e-3, (0.9, 0.999), 1e-8, 0.01, None)
            for ts in zip(p, g, m, v)]
    old = [t.cpu().double() for t in p]
    ops.adamw_step(p, g, m, v, 3)
    assert ops.launch_count() >= 2
    for k in range(count):
        check_p(p[k], want[k][0], want[k][0] - old[k])


def test_tensors_without_a_gradient_stay(ops):
    p, g, m, v = make([(100,), (50,), (64,)])
    old = [t.clone() for t in (p[1], m[1], v[1])]
    g[1] = None
    ops.adamw_step(p, g, m, v, 1)
    assert all(torch.equal(a, b) for a, b in zip(old, (p[1], m[1], v[1])))
    ops.adamw_step([], [], [], [], 1)
    assert ops.status() == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_follows_its_counter(ops, bits):
    def fresh():
        p, g, m, v = make([(300,), (64, 65)], seed=8)
        if bits == 8:
            m, v = ([ops.state8_pack(t, s) for t in ts] for ts, s in ((m, True), (v, False)))
        return p, g, m, v

    def values(ts):
        return [u for t in ts for u in (t if isinstance(t, tuple) else (t,))]
    p, g, m, v = fresh()
    for step, lr in ((4, 1e-2), (5, 5e-3), (6, 2e-3)):
        ops.adamw_step(p, g, m, v, step, lr=lr, seed=2)
    q, g2, m2, v2 = fresh()
    step, rate = torch.tensor([4], dtype=torch.int32, device="cuda"), torch.tensor([1e-2], device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.adamw_step(q, g2, m2, v2, step, lr=rate, seed=2)
    for t, lr in ((4, 1e-2), (5, 5e-3), (6, 2e-3)):
        step.fill_(t)
        rate.fill_(lr)
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(values(m) + values(v), values(m2) + values(v2)):
        assert torch.equal(a, b)
    for a, b in zip(p, q):  # lr in fp32: a rounding of the update
        assert float((a - b).abs().max()) <= 1e-6


def test_refusals(ops):
    p, g, m, v = make([(64,), (10,)])
    m8, v8 = [ops.state8_pack(t, True) for t in m], [ops.state8_pack(t, False) for t in v]
    bad = [
        (p, g[:1], m, v), (p, [g[0], g[1].double()], m, v), (p, [g[0], g[1][:9]], m, v), (p, g, m8, v),
        (p, g, m, v8), ([p[0].cpu(), p[1]], g, m, v), ([p[0], torch.zeros(20, device="cuda")[::2]], g, m, v),
        (p, g, [m[0], m[1].bfloat16()], v), (p, g, [m8[0], (m8[1][0], m8[0][1][:0])], v8)]
    for args in bad:
        with pytest.raises(ValueError):
            ops.adamw_step(*args, 1)
    for kw in ({"betas": (1.0, 0.9)}, {"betas": (0.9, -0.1)}, {"eps": -1.0}, {"lr": float("nan")},
               {"weight_decay": float("inf")}):
        with pytest.raises(binding.RcuError):
            ops.adamw_step(p, g, m, v, 1, **kw)
    with pytest.raises(binding.RcuError):
        ops.adamw_step(p, g, m, v, 0)
    with pytest.raises(ValueError):
        ops.adamw_step(p, g, m, v, 1, scale=0.5)
    with pytest.raises(binding.RcuError):  # a bf16 parameter needs no copy
        ops.adamw_step([t.bfloat16() for t in p], g, m, v, 1, copies=[t.bfloat16() for t in p])
