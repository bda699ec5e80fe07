"""The sequence operators' cases: a gated linear recurrence (forward, backward,
single-token step), layer norm (forward, backward) and 8-bit activation
checkpoints (alone, and in the two backward passes).

`run` computes one pass of a case, either in plain torch operations in 32 bits
(own = False) or through the framework's public calls (own = True); `exact`
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64   # steps between the states that the forward keeps for the backward
BLOCK = 64   # values that share an exponent in an 8-bit checkpoint
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

_handle = None


def _ops():
    """The framework's handle, made once as a user's program would."""
    global _handle
    if _handle is None:
        from recurrent_cell_unroll_gb300 import binding
        _handle = binding.SeqOps()
    return _handle


# --------------------------------------------------------------------------- cases

def _rec(op, T, B, H, dtype, varlen=False, batch_first=False, act8=False):
    return {"op": op, "T": T, "B": B, "H": H, "dtype": dtype, "varlen": varlen,
            "batch_first": batch_first, "act8": act8}


def _ln(op, rows, n, dtype, residual=False, act8=False):
    return {"op": op, "rows": rows, "n": n, "dtype": dtype, "residual": residual, "act8": act8}


def listed():
    return [
        # one short sequence: the framework's smallest forward shape, where latency counts
        dict(_rec("rec_fwd", 80, 1, 256, "f32"), name="rec_fwd_f32_T80_B1_H256"),
        # a training batch of the framework's largest stacked shape
        dict(_rec("rec_fwd", 512, 256, 1024, "bf16"), name="rec_fwd_bf16_T512_B256_H1024"),
        # prefill of one long sequence: few channels, so time has to be split
        dict(_rec("rec_fwd", 65536, 1, 2048, "bf16"), name="rec_fwd_bf16_T65536_B1_H2048"),
        # training on a padded batch of the framework's variable-length shape
        dict(_rec("rec_bwd", 500, 64, 512, "f32", varlen=True), name="rec_bwd_f32_varlen_T500_B64_H512"),
        # training on a few long sequences, batch-major
        dict(_rec("rec_bwd", 8192, 4, 2048, "bf16", batch_first=True), name="rec_bwd_bf16_T8192_B4_H2048"),
        # training with the recurrence's inputs kept in 8 bits
        dict(_rec("rec_bwd", 1000, 32, 1024, "bf16", act8=True), name="rec_bwd_act8_T1000_B32_H1024"),
        # serving: one token of every running request, states in a table of slots
        dict(_rec("rec_step", 1, 256, 1024, "bf16"), name="rec_step_bf16_B256_H1024"),
        # a small normalisation beside the framework's smallest cells
        dict(_ln("ln_fwd", 50, 200, "f32"), name="ln_fwd_f32_50x200"),
        # the normalisation between two layers of the largest stacked shape, with the residual
        dict(_ln("ln_fwd", 131072, 1024, "bf16", residual=True), name="ln_fwd_bf16_131072x1024"),
        # and its backward pass
        dict(_ln("ln_bwd", 131072, 1024, "bf16", residual=True), name="ln_bwd_bf16_131072x1024"),
        # a backward pass from an 8-bit checkpoint, a width that is no multiple of its blocks
        dict(_ln("ln_bwd", 12501, 1000, "f32", act8=True), name="ln_bwd_act8_f32_12501x1000"),
        # writing a checkpoint and reading it back
        dict(_ln("act8", 32768, 2048, "bf16"), name="act8_bf16_32768x2048"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 8, as most models have, half of any size."""
    n = _log(rng, lo, hi)
    return max(8, n // 8 * 8) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["rec_fwd", "rec_fwd", "rec_bwd", "rec_bwd", "rec_step", "ln_fwd", "ln_bwd", "act8"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "rec_step":
        return _rec(op, 1, _log(rng, 1, 1024), _width(rng, 64, 4096), dtype)
    if op.startswith("rec"):
        T, B, H = _log(rng, 1, 65536), _log(rng, 1, 256), _width(rng, 64, 4096)
        T = max(1, min(T, (1 << 25) // (B * H)))
        return _rec(op, T, B, H, dtype, varlen=rng.random() < 0.3, batch_first=rng.random() < 0.3,
                    act8=op == "rec_bwd" and rng.random() < 0.3)
    n = _width(rng, 64, 8192)
    rows = max(1, min(_log(rng, 1, 131072), (1 << 26) // n))
    return _ln(op, rows, n, dtype, residual=op != "act8" and rng.random() < 0.5,
               act8=op == "ln_bwd" and rng.random() < 0.3)


def _size(dtype):
    return DTYPES[dtype].itemsize


def work(case):
    """Each input read once and each output written once; operations counted
    per element (an exponential, a root or a division as one)."""
    e = _size(case["dtype"])
    if case["op"].startswith("rec"):
        T, B, H = case["T"], case["B"], case["H"]
        n, chunks = T * B * H, -(-T // CHUNK)
        small = 4 * H * (2 + 2 * B)
        live = (T // 10 + T) / (2 * T) if case["varlen"] else 1  # the share of steps that are read
        if case["op"] == "rec_step":
            return {"bytes": n * (4 * e + 8) + 4 * H + 4 * B, "flops": 18.0 * n}
        kept = 4 * chunks * B * H
        if case["op"] == "rec_fwd":
            return {"bytes": n * e * (3 * live + 1) + kept + small, "flops": 18.0 * n * live}
        saved = (1 + 1 / BLOCK) if case["act8"] else e
        return {"bytes": n * (live * (3 * saved + e) + 3 * e) + kept + small, "flops": 45.0 * n * live}
    n, rows = case["rows"] * case["n"], case["rows"]
    if case["op"] == "ln_fwd":
        return {"bytes": n * e * (4 if case["residual"] else 2) + 8 * rows + 8 * case["n"], "flops": 8.0 * n}
    if case["op"] == "ln_bwd":
        saved = (1 + 1 / BLOCK) if case["act8"] else e
        return {"bytes": n * (saved + e * (3 if case["residual"] else 2)) + 8 * rows + 12 * case["n"],
                "flops": 16.0 * n}
    return {"bytes": n * 2 * (e + 1 + 1 / BLOCK), "flops": 6.0 * n}


# --------------------------------------------------------------------------- plain forms, 32 bits

def _scan(a, b, h0):
    """h_t = a_t h_{t-1} + b_t along the first dimension, by doubling."""
    b = torch.cat([(b[0] + a[0] * h0)[None], b[1:]])
    d = 1
    while d < a.shape[0]:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _time_first(t, case):
    return t.transpose(0, 1) if case["batch_first"] else t


def _mask(case, lengths, device):
    """[T, B, 1]: the steps that take part."""
    t = torch.arange(case["T"], device=device)[:, None]
    if lengths is None:
        return (t >= 0).expand(case["T"], case["B"])[..., None]
    return (t < lengths[None, :])[..., None]


def _gates(x, r, i, lam, c):
    s, g = torch.sigmoid(r), torch.sigmoid(i)
    k = c * torch.log1p(torch.exp(lam))
    a = torch.exp(-k * s)
    w = -torch.expm1(-2 * k * s)
    return s, g, k, a, w


def _power(e):
    """2^e in 32 bits, exactly, for whole e between -126 and 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _values8(codes, exps, n):
    """What an 8-bit checkpoint stands for, in 32 bits."""
    return codes.float() * _power(exps).repeat_interleave(BLOCK, -1)[..., :n]


def _codes8(v):
    """(codes, exponents) of an 8-bit checkpoint of v (finite values)."""
    n = v.shape[-1]
    blocks = torch.nn.functional.pad(v.float(), (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = blocks.abs().amax(-1)
    m, q = torch.frexp(top)
    e = torch.where(m * 128 <= 127, q - 7, q - 6)
    e = torch.where(top > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    codes = torch.round(blocks * _power(-e)[..., None])
    return codes.flatten(-2)[..., :n].to(torch.int8), e.to(torch.int8)


def _rec_fwd(case, st):
    x, r, i = (_time_first(st[k], case).float() for k in ("x", "r", "i"))
    keep = _mask(case, st["lengths"], x.device)
    s, g, _, a, w = _gates(x, r, i, st["lam"], st["c"])
    a = torch.where(keep, a, torch.ones_like(a))
    b = torch.where(keep, torch.sqrt(w) * g * x, torch.zeros_like(a))
    h = _scan(a, b, st["h0"])
    y = torch.where(keep, h, torch.zeros_like(h)).to(st["x"].dtype)
    states = torch.cat([st["h0"][None], h[CHUNK - 1:-1:CHUNK]])
    return _time_first(y, case), h[-1], states


def _saved(case, st, k):
    return _values8(*st[k], case["H"]) if case["act8"] else st[k].float()


def _rec_bwd(case, st):
    T, B, H = case["T"], case["B"], case["H"]
    x, r, i = (_time_first(_saved(case, st, k), case) for k in ("x", "r", "i"))
    dy = _time_first(st["dy"], case).float()
    keep = _mask(case, st["lengths"], dy.device)
    s, g, k, a, w = _gates(x, r, i, st["lam"], st["c"])
    one, zero = torch.ones_like(a), torch.zeros_like(a)
    beta = torch.sqrt(w)
    b = torch.where(keep, beta * g * x, zero)
    a1 = torch.where(keep, a, one)
    # the states before each step, from the kept ones: every chunk at once
    chunks = -(-T // CHUNK)
    pad = (0, 0, 0, 0, 0, chunks * CHUNK - T)
    ac = torch.nn.functional.pad(a1, pad, value=1.0).view(chunks, CHUNK, B, H).transpose(0, 1)
    bc = torch.nn.functional.pad(b, pad).view(chunks, CHUNK, B, H).transpose(0, 1)
    h = torch.cat([st["states"][None], _scan(ac, bc, st["states"])[:-1]])
    h = h.transpose(0, 1).reshape(chunks * CHUNK, B, H)[:T]
    # the gradient reaching each state, backwards in time
    nxt = torch.cat([a1[1:], one[:1]])
    e = _scan(nxt.flip(0), torch.where(keep, dy, zero).flip(0), st["dh_n"]).flip(0)
    dlog = torch.where(keep, e * (a * h - a * a / beta * (g * x)), zero)
    dx = torch.where(keep, e * beta * g, zero)
    di = torch.where(keep, e * beta * g * (1 - g) * x, zero)
    dr = -k * dlog * s * (1 - s)
    dlam = -st["c"] * torch.sigmoid(st["lam"]) * (dlog * s).sum((0, 1))
    out = [_time_first(v.to(st["dy"].dtype), case) for v in (dx, dr, di)]
    return (*out, dlam, a1[0] * e[0])


def _rec_step(case, st):
    x, r, i = (st[k].float() for k in ("x", "r", "i"))
    s, g, _, a, w = _gates(x, r, i, st["lam"], st["c"])
    slot = st["slot"].long()
    h = a * st["state"][slot] + torch.sqrt(w) * g * x
    st["state"][slot] = h
    return h.to(st["x"].dtype), st["state"]


def _ln_fwd(case, st):
    u = st["x"].float()
    if case["residual"]:
        u = (u + st["residual"].float()).to(st["x"].dtype).float()
    mean = u.mean(-1)
    d = u - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(-1) + st["eps"])
    y = (d * rstd[:, None] * st["weight"] + st["bias"]).to(st["x"].dtype)
    return (y, u.to(st["x"].dtype), mean, rstd) if case["residual"] else (y, mean, rstd)


def _ln_bwd(case, st):
    u = _values8(*st["x"], case["n"]) if case["act8"] else st["x"].float()
    dy = st["dy"].float()
    xh = (u - st["mean"][:, None]) * st["rstd"][:, None]
    q = dy * st["weight"]
    du = st["rstd"][:, None] * (q - q.mean(-1, keepdim=True) - xh * (q * xh).mean(-1, keepdim=True))
    if case["residual"]:
        du = du + st["dsum"].float()
    return du.to(st["dy"].dtype), (dy * xh).sum(0), dy.sum(0)


def _act8(case, st):
    return _values8(*_codes8(st["x"]), case["n"]).to(st["x"].dtype)


PLAIN = {"rec_fwd": _rec_fwd, "rec_bwd": _rec_bwd, "rec_step": _rec_step, "ln_fwd": _ln_fwd,
         "ln_bwd": _ln_bwd, "act8": _act8}


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32, std=1.0):
        # filled in parts: no 32-bit copy of a large 16-bit tensor is needed at once
        out = torch.empty(shape, device=dev, dtype=dtype)
        for part in out.flatten().split(1 << 26):
            part.copy_(torch.randn(part.shape, generator=g, device=dev) * std)
        return out

    if not case["op"].startswith("rec"):
        rows, n = case["rows"], case["n"]
        st = {"weight": 1 + normal(n, std=0.1), "bias": normal(n, std=0.1), "eps": 1e-5}
        # a residual stream: a channel mean and scale of its own on every value
        x = (normal(rows, n, dtype=dt) * (0.5 + torch.rand(n, generator=g, device=dev)).to(dt)
             + normal(n, std=0.2).to(dt))
        st["x"] = x
        if case["op"] == "ln_fwd" and case["residual"]:
            st["residual"] = normal(rows, n, dtype=dt)
        if case["op"] == "ln_bwd":
            st["mean"] = torch.cat([p.float().mean(-1) for p in x.split(1 << 14)])
            var = torch.cat([p.float().var(-1, correction=0) for p in x.split(1 << 14)])
            st["rstd"] = 1 / torch.sqrt(var + st["eps"])
            st["dy"] = normal(rows, n, dtype=dt)
            if case["residual"]:
                st["dsum"] = normal(rows, n, dtype=dt)
            if case["act8"]:
                st["x"] = _codes8(x)
        st["case"] = case
        return st

    T, B, H = case["T"], case["B"], case["H"]
    st = {"c": 8.0, "case": case}
    # decays that remember between about ten and a thousand steps at an open gate
    top = 0.9 + 0.099 * torch.rand(H, generator=g, device=dev)
    st["lam"] = torch.log(torch.expm1(-torch.log(top) / st["c"]))
    if case["op"] == "rec_step":
        shape = (B, H)
        slots = 2 * B
        st["state"] = normal(slots, H, std=0.5)
        st["slot"] = torch.randperm(slots, generator=g, device=dev)[:B].to(torch.int32)
    else:
        shape = (B, T, H) if case["batch_first"] else (T, B, H)
        st["h0"] = normal(B, H, std=0.5)
        st["lengths"] = (torch.randint(T // 10, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
                         if case["varlen"] else None)
    for k in ("x", "r", "i"):
        st[k] = normal(*shape, dtype=dt)
    if case["op"] == "rec_bwd":
        _, st["h_n"], st["states"] = _rec_fwd(case, st)
        st["dy"] = normal(*shape, dtype=dt)
        st["dh_n"] = normal(B, H)
        if case["act8"]:
            for k in ("x", "r", "i"):
                st[k] = _codes8(st[k])
    return st


# --------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if not own:
        return PLAIN[case["op"]](case, st)
    ops = _ops()
    if case["op"] == "rec_fwd":
        return ops.linrec_forward(st["x"], st["r"], st["i"], st["lam"], c=st["c"], lengths=st["lengths"],
                                  h0=st["h0"], batch_first=case["batch_first"], states=True)
    if case["op"] == "rec_bwd":
        return ops.linrec_backward(st["dy"], st["x"], st["r"], st["i"], st["lam"], st["states"], c=st["c"],
                                   lengths=st["lengths"], dh_n=st["dh_n"], batch_first=case["batch_first"])
    if case["op"] == "rec_step":
        return ops.linrec_step(st["x"], st["r"], st["i"], st["lam"], st["state"], c=st["c"],
                               slot=st["slot"]), st["state"]
    if case["op"] == "ln_fwd":
        if case["residual"]:
            return ops.layernorm_forward(st["x"], st["weight"], st["bias"], eps=st["eps"],
                                         residual=st["residual"])
        return ops.layernorm_forward(st["x"], st["weight"], st["bias"], eps=st["eps"])
    if case["op"] == "ln_bwd":
        return ops.layernorm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["weight"],
                                      dsum=st.get("dsum"))
    return ops.act8_unpack(*ops.act8_pack(st["x"]), dtype=st["x"].dtype)


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)

    def power(e):  # 2^e in 64 bits, exactly
        return ((e.long() + 1023) << 52).view(torch.float64)

    def wide(t):
        if isinstance(t, tuple):
            codes, exps = t
            n = codes.shape[-1]
            at = torch.arange(n, device=codes.device) // BLOCK
            return codes.double() * power(exps)[..., at]
        return t.double()

    if case["op"] == "act8":
        v = wide(st["x"])
        out = torch.empty_like(v)
        for k in range(0, case["n"], BLOCK):
            b = v[:, k:k + BLOCK]
            top = b.abs().amax(1, keepdim=True)
            # the smallest power of two of which 127 times reach the largest value
            e = torch.ceil(torch.log2(top / 127)).clamp(min=-126)
            e = torch.where(127 * power(e - 1) >= top, e - 1, e)
            e = torch.where(127 * power(e) < top, e + 1, e).clamp(min=-126)
            out[:, k:k + BLOCK] = torch.round(b / power(e)) * power(e)
        return out
    if case["op"].startswith("ln"):
        u = wide(st["x"])
        if case["op"] == "ln_fwd":
            if case["residual"]:
                u = (st["x"].float() + st["residual"].float()).to(st["x"].dtype).double()
            var, mean = torch.var_mean(u, -1, correction=0)
            rstd = (var + st["eps"]) ** -0.5
            y = (u - mean[:, None]) * rstd[:, None] * st["weight"].double() + st["bias"].double()
            return (y, u, mean, rstd) if case["residual"] else (y, mean, rstd)
        dy, weight = wide(st["dy"]), wide(st["weight"])
        xh = (u - wide(st["mean"])[:, None]) * wide(st["rstd"])[:, None]
        dxh = dy * weight
        n = case["n"]
        du = (n * dxh - dxh.sum(1, keepdim=True) - xh * (dxh * xh).sum(1, keepdim=True)) / n
        du = du * wide(st["rstd"])[:, None] + (wide(st["dsum"]) if case["residual"] else 0)
        return du, (dy * xh).sum(0), dy.sum(0)

    lam, c = wide(st["lam"]), st["c"]
    rate = c * torch.nn.functional.softplus(lam, threshold=1e6)
    x, r, i = (wide(st[k]) for k in ("x", "r", "i"))
    if case["op"] != "rec_step" and case["batch_first"]:
        x, r, i = (t.transpose(0, 1) for t in (x, r, i))
    s, gate = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    a = torch.exp(-rate * s)
    beta = torch.sqrt(-torch.expm1(-2 * rate * s))
    if case["op"] == "rec_step":
        h = a * wide(st["state"])[st["slot"].long()] + beta * gate * x
        state = wide(st["state"]).clone()
        state[st["slot"].long()] = h
        return h, state

    T, B, H = case["T"], case["B"], case["H"]
    steps = torch.arange(T, device=x.device)[:, None, None]
    ends = torch.full((B,), T, device=x.device) if st["lengths"] is None else st["lengths"]
    dead = steps >= ends[None, :, None]
    if case["op"] == "rec_fwd":
        a.masked_fill_(dead, 1)
        b = (beta * gate * x).masked_fill_(dead, 0)
        h, states = wide(st["h0"]), []
        for t in range(T):  # one step after another
            if t % CHUNK == 0:
                states.append(h)
            h = torch.addcmul(b[t], a[t], h, out=b[t])
        h_n = h.clone()
        states = torch.stack(states)
        y = b.masked_fill_(dead, 0)
        return (y.transpose(0, 1) if case["batch_first"] else y), h_n, states

    dy = wide(st["dy"])
    dy = dy.transpose(0, 1) if case["batch_first"] else dy
    b = beta * gate * x
    before = torch.empty_like(a)  # the state before each step
    for t in range(T):
        h = wide(st["states"][t // CHUNK]) if t % CHUNK == 0 else torch.addcmul(b[t - 1], a[t - 1], h)
        h = torch.where(dead[t], torch.zeros_like(h), h)
        before[t] = h
    e, come = torch.empty_like(a), wide(st["dh_n"])
    for t in reversed(range(T)):  # the gradient reaching each state
        e[t] = torch.where(dead[t], torch.zeros_like(come), dy[t] + come)
        come = torch.where(dead[t], come, a[t] * e[t])
    dlog = e * (a * before - a * a * gate * x / beta)
    dx, di = e * beta * gate, e * beta * x * gate * (1 - gate)
    dr = -rate * dlog * s * (1 - s)
    dlam = -c / (1 + torch.exp(-lam)) * (dlog * s).sum((0, 1))
    out = [v.transpose(0, 1) if case["batch_first"] else v for v in (dx, dr, di)]
    return (*out, dlam, come)
