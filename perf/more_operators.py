"""Cases of a selective state space scan and its short causal convolution (forward,
backward, single tokens), and of an AdamW step over many tensors with states in
32 or in 8 bits.

`run` computes one pass of a case, either in plain torch operations in 32 bits
(own = False) or through the framework's public calls (own = True); `exact`
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK = 32   # steps between the states that the scan's forward keeps for its backward
BLOCK = 64   # values that share an exponent in an 8-bit optimizer state
# an 8-bit state's code counts eighths of octaves above an offset: 2^-14 of the block's
# power of two in the signed first moment, 2^-30 in the unsigned second one
OCTAVES = {"m": 14, "v": 30}
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

def _conv(op, T, B, H, W, dtype, varlen=False, batch_first=False):
    return {"op": op, "T": T, "B": B, "H": H, "W": W, "dtype": dtype, "varlen": varlen,
            "batch_first": batch_first}


def _ssm(op, T, B, H, N, dtype, varlen=False, batch_first=False, train=False):
    return {"op": op, "T": T, "B": B, "H": H, "N": N, "dtype": dtype, "varlen": varlen,
            "batch_first": batch_first, "train": train}


def _token(B, H, N, W, dtype):
    return {"op": "token", "B": B, "H": H, "N": N, "W": W, "dtype": dtype}


def _adamw(layers, dim, hidden, bits, grad, scaled=False):
    return {"op": "adamw", "layers": layers, "dim": dim, "hidden": hidden, "bits": bits, "grad": grad,
            "scaled": scaled}


def listed():
    return [
        # one short sequence of a small model, where latency counts
        dict(_conv("conv_fwd", 80, 1, 256, 4, "f32"), name="conv_fwd_f32_T80_B1_H256"),
        # a training batch of the framework's largest stacked shape
        dict(_conv("conv_fwd", 512, 256, 1024, 4, "bf16"), name="conv_fwd_bf16_T512_B256_H1024"),
        # training on a padded batch of the framework's variable-length shape
        dict(_conv("conv_bwd", 500, 64, 512, 4, "f32", varlen=True), name="conv_bwd_f32_varlen_T500_B64_H512"),
        # training on a few long sequences, batch-major
        dict(_conv("conv_bwd", 8192, 4, 2048, 4, "bf16", batch_first=True), name="conv_bwd_bf16_T8192_B4_H2048"),
        # the forward pass of a training step, which keeps states for the backward pass
        dict(_ssm("scan_fwd", 2048, 8, 2048, 16, "bf16", train=True), name="scan_fwd_bf16_T2048_B8_H2048"),
        # the prompt of one long sequence: few channels, so time has to be split
        dict(_ssm("scan_fwd", 65536, 1, 512, 16, "bf16", batch_first=True), name="scan_fwd_bf16_T65536_B1_H512"),
        # training on a padded batch in full precision
        dict(_ssm("scan_bwd", 500, 32, 512, 16, "f32", varlen=True), name="scan_bwd_f32_varlen_T500_B32_H512"),
        # training on a few long sequences, batch-major
        dict(_ssm("scan_bwd", 8192, 2, 1024, 16, "bf16", batch_first=True), name="scan_bwd_bf16_T8192_B2_H1024"),
        # serving one request, where latency counts
        dict(_token(1, 512, 16, 4, "f32"), name="token_f32_B1_H512"),
        # serving: one token of every running request, states in tables of slots
        dict(_token(256, 2048, 16, 4, "bf16"), name="token_bf16_B256_H2048"),
        # the optimizer step of a stack of 24 such blocks, states in full precision
        dict(_adamw(24, 1024, 2048, 32, "f32"), name="adamw32_24x1024x2048"),
        # the same with states in 8 bits, odd widths, and gradients in bf16 that are clipped
        dict(_adamw(8, 1000, 2001, 8, "bf16", scaled=True), name="adamw8_8x1000x2001"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 8, as most models have, half of any size."""
    n = _log(rng, lo, hi)
    return max(8, n // 8 * 8) if rng.random() < 0.5 else n


def _states(rng):
    return rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)])


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "token", "adamw"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "token":
        return _token(_log(rng, 1, 1024), _width(rng, 64, 4096), _states(rng), rng.randint(2, 4), dtype)
    if op == "adamw":
        dim, layers = _width(rng, 64, 2048), _log(rng, 1, 48)
        layers = max(1, min(layers, (1 << 27) // (7 * dim * dim)))
        return _adamw(layers, dim, rng.choice([dim, 2 * dim]), rng.choice([8, 32]), dtype, rng.random() < 0.5)
    T, B, H = _log(rng, 1, 65536), _log(rng, 1, 256), _width(rng, 64, 4096)
    flags = {"varlen": rng.random() < 0.3, "batch_first": rng.random() < 0.3}
    if op.startswith("conv"):
        T = max(1, min(T, (1 << 25) // (B * H)))
        return _conv(op, T, B, H, rng.randint(2, 4), dtype, **flags)
    N = _states(rng)
    T = max(1, min(T, (1 << (29 if op == "scan_fwd" else 28)) // (B * H * N)))
    return _ssm(op, T, B, H, N, dtype, train=op == "scan_fwd" and rng.random() < 0.5, **flags)


def _shapes(case):
    """The parameters of a stack of blocks: norm, projections, convolution, scan."""
    dim, hid, N, rank = case["dim"], case["hidden"], 16, -(-case["dim"] // 16)
    block = [(dim,), (dim,), (dim, 2 * hid), (hid, 4), (hid,), (hid, rank + 2 * N), (rank, hid), (hid,),
             (hid, N), (hid,), (hid, dim)]
    return block * case["layers"]


def work(case):
    """Each input read once and each output written once; operations counted
    per element (an exponential, a root or a division as one)."""
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        grad = DTYPES[case["grad"]].itemsize
        # in 8 bits the pass also reads both states out in 32 bits
        held = 16 if case["bits"] == 32 else 4 * (1 + 1 / BLOCK) + 2 * (1 + 1 / BLOCK + 4)
        return {"bytes": n * (8 + grad + held), "flops": (12.0 if case["bits"] == 32 else 50.0) * n}
    e = DTYPES[case["dtype"]].itemsize
    B, H = case["B"], case["H"]
    if case["op"] == "token":
        N, W = case["N"], case["W"]
        conv = B * H * e * (2 + 2 * (W - 1)) + 4 * H * (W + 1)
        scan = B * H * (4 * e + 8 * N) + 2 * B * N * e + 4 * H * (N + 2)
        return {"bytes": conv + scan + 8 * B, "flops": B * H * (2.0 * W + 6 + 7 * N)}
    T = case["T"]
    n = T * B * H
    live = (T // 10 + T) / (2 * T) if case["varlen"] else 1  # the share of steps that are read
    if case["op"] == "conv_fwd":
        return {"bytes": n * e * (live + 1) + 4 * H * (case["W"] + 1) + 2 * e * B * H * (case["W"] - 1),
                "flops": (2.0 * case["W"] + 6) * n * live}
    if case["op"] == "conv_bwd":
        return {"bytes": n * e * (2 * live + 1) + 8 * H * (case["W"] + 1) + 2 * e * B * H * (case["W"] - 1),
                "flops": (6.0 * case["W"] + 10) * n * live}
    N = case["N"]
    kept, small = 4 * -(-T // CHUNK) * B * H * N, 4 * H * (N + 2) + 8 * B * H * N
    if case["op"] == "scan_fwd":
        return {"bytes": n * e * (3 * live + 1) + 2 * T * B * N * e * live + small + (kept if case["train"] else 0),
                "flops": n * live * (7.0 * N + 14)}
    return {"bytes": n * e * (4 * live + 3) + 2 * T * B * N * e * (live + 1) + kept + 2 * small,
            "flops": n * live * (21.0 * N + 40)}


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


def _keep(case, lengths, device):
    """[T, B, 1]: the steps that take part."""
    t = torch.arange(case["T"], device=device)[:, None]
    if lengths is None:
        return (t >= 0).expand(case["T"], case["B"])[..., None]
    return (t < lengths[None, :])[..., None]


def _silu(v):
    return v / (1 + torch.exp(-v))


def _silu_slope(v):
    s = 1 / (1 + torch.exp(-v))
    return s * (1 + v * (1 - s))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _conv_in(case, st):
    """The inputs with the state before them, [T + W - 1, B, H], 0 past a row's end."""
    x = _time_first(st["x"], case).float()
    x = torch.where(_keep(case, st["lengths"], x.device), x, torch.zeros_like(x))
    return torch.cat([st["state"].float().transpose(0, 1), x])


def _taps(case, st, x):
    return sum((st["weight"][:, k] * x[k:k + case["T"]] for k in range(case["W"])), st["bias"])


def _conv_fwd(case, st):
    T, W = case["T"], case["W"]
    x = _conv_in(case, st)
    y = _silu(_taps(case, st, x))
    y = torch.where(_keep(case, st["lengths"], x.device), y, torch.zeros_like(y)).to(st["x"].dtype)
    end = torch.full((case["B"],), T, device=x.device) if st["lengths"] is None else st["lengths"]
    at = end[:, None] + torch.arange(W - 1, device=x.device)[None, :]
    state = x[at.long(), torch.arange(case["B"], device=x.device)[:, None]]
    return _time_first(y, case), state.to(st["x"].dtype)


def _conv_bwd(case, st):
    T, W = case["T"], case["W"]
    x = _conv_in(case, st)
    dy = _time_first(st["dy"], case).float()
    dv = dy * _silu_slope(_taps(case, st, x))
    dv = torch.where(_keep(case, st["lengths"], x.device), dv, torch.zeros_like(dv))
    wide = torch.nn.functional.pad(dv, (0, 0, 0, 0, W - 1, W - 1))
    dx = sum(st["weight"][:, k] * wide[W - 1 - k:W - 1 - k + T + W - 1] for k in range(W))
    dw = torch.stack([(dv * x[k:k + T]).sum((0, 1)) for k in range(W)], 1)
    dtype = st["x"].dtype
    keep = _keep(case, st["lengths"], x.device)
    dstate, dx = dx[:W - 1].transpose(0, 1), torch.where(keep, dx[W - 1:], torch.zeros_like(dv))
    return _time_first(dx.to(dtype), case), dw, dv.sum((0, 1)), dstate.to(dtype)


def _scan_in(case, st):
    """x, delta, keep [T, B, H], a and delta x B [T, B, H, N], steps past a row's end left out."""
    x, dt = (_time_first(st[k], case).float() for k in ("x", "dt"))
    keep = _keep(case, st["lengths"], x.device)
    zero = torch.zeros_like(x)
    x = torch.where(keep, x, zero)
    delta = torch.where(keep, _softplus(dt + st["dt_bias"]), zero)
    a = torch.exp(delta[..., None] * -torch.exp(st["a_log"]))
    b = torch.where(keep, _time_first(st["b"], case).float(), torch.zeros_like(delta[..., :1]))
    return x, dt, delta, keep, a, b, (delta * x)[..., None] * b[:, :, None]


def _scan_fwd(case, st):
    x, _, _, keep, a, _, u = _scan_in(case, st)
    h = _scan(a, u, st["h0"])
    c, z = (_time_first(st[k], case).float() for k in ("c", "z"))
    y = ((h * c[:, :, None]).sum(-1) + st["d"] * x) * _silu(z)
    y = torch.where(keep, y, torch.zeros_like(y)).to(st["x"].dtype)
    out = [_time_first(y, case), h[-1].clone()]
    return out + [torch.cat([st["h0"][None], h[CHUNK - 1:-1:CHUNK]])] if case["train"] else out


def _scan_bwd(case, st):
    T, B, H, N = case["T"], case["B"], case["H"], case["N"]
    x, dt, delta, keep, a, b, u = _scan_in(case, st)
    zero = torch.zeros_like(x)
    # the states before each step, from the kept ones: every chunk at once
    chunks = -(-T // CHUNK)
    pad = (0, 0, 0, 0, 0, 0, 0, chunks * CHUNK - T)
    ac = torch.nn.functional.pad(a, pad, value=1.0).view(chunks, CHUNK, B, H, N).transpose(0, 1)
    uc = torch.nn.functional.pad(u, pad).view(chunks, CHUNK, B, H, N).transpose(0, 1)
    h = _scan(ac, uc, st["states"])
    before = torch.cat([st["states"][None], h[:-1]]).transpose(0, 1).reshape(chunks * CHUNK, B, H, N)[:T]
    h = h.transpose(0, 1).reshape(chunks * CHUNK, B, H, N)[:T]
    c, z, dy = (_time_first(st[k], case).float() for k in ("c", "z", "dy"))
    s = (h * c[:, :, None]).sum(-1) + st["d"] * x
    dz = torch.where(keep, dy * s * _silu_slope(z), zero)
    gy = torch.where(keep, dy * _silu(z), zero)
    c = torch.where(keep, c, torch.zeros_like(c))
    dc = (gy[..., None] * h).sum(2)
    # the gradient reaching each state, backwards in time
    nxt = torch.cat([a[1:], torch.ones_like(a[:1])])
    e = _scan(nxt.flip(0), (gy[..., None] * c[:, :, None]).flip(0), st["dh_n"]).flip(0)
    du = (e * b[:, :, None]).sum(-1)
    dlog = e * a * before * -torch.exp(st["a_log"])
    ddt = torch.where(keep, (dlog.sum(-1) + du * x) / (1 + torch.exp(-(dt + st["dt_bias"]))), zero)
    dx = torch.where(keep, du * delta + gy * st["d"], zero)
    db = (e * (delta * x)[..., None]).sum(2)
    out = [_time_first(v.to(st["x"].dtype), case) for v in (dx, ddt, db, dc, dz)]
    return (*out, (dlog * delta[..., None]).sum((0, 1)), (gy * x).sum((0, 1)), ddt.sum((0, 1)), a[0] * e[0])


def _token_fwd(case, st):
    """The convolution's step, then the scan's, each with states in a table."""
    slot = st["slot"].long()
    xs = torch.cat([st["window"][slot].float(), st["x"].float()[:, None]], 1)
    u = _silu((xs * st["weight"].t()).sum(1) + st["bias"])
    st["window"][slot] = xs[:, 1:].to(st["x"].dtype)
    x, dt, b, c, z = (st[k].float() for k in ("xs", "dt", "b", "c", "z"))
    delta = _softplus(dt + st["dt_bias"])
    h = torch.exp(delta[..., None] * -torch.exp(st["a_log"])) * st["states"][slot] \
        + (delta * x)[..., None] * b[:, None]
    st["states"][slot] = h
    y = ((h * c[:, None]).sum(-1) + st["d"] * x) * _silu(z)
    return u.to(st["x"].dtype), st["window"], y.to(st["x"].dtype), st["states"]


# 8-bit optimizer states.  A block of 64 values has a power of two 2^e, that of its
# largest finite magnitude (e between -126 and 126).  With f = |v| 2^-e and an offset
# o = 2^-OCTAVES, f + o is rounded to three bits behind its leading one, up or down by
# the element's random bits, and its code counts such steps above o.  The first moment's
# code is an int8 with the sign; the second's a whole number up to 254 less 128, and at least one step for a v above 0.

def _power(e):
    """2^e in 32 bits, exactly, for whole e between -126 and 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _state8_values(codes, exps, kind):
    """What codes [..., 64] with exponents [...] stand for, in 32 bits."""
    o = OCTAVES[kind]
    q = codes.int()
    n = q.abs() if kind == "m" else q + 128
    v = ((n + ((127 - o) << 3)) << 20).view(torch.float32) - 2.0 ** -o
    v = torch.where(q < 0, -v, v) if kind == "m" else v
    return v * _power(exps)[..., None]


def _state8_codes(v, bits, kind):
    """(codes, exponents) of blocks v [..., 64] (finite), rounded by 16 random bits each."""
    o = OCTAVES[kind]
    e = ((v.abs().amax(-1).view(torch.int32) >> 23) - 127).clamp(-126, 126)
    f = v.abs() * _power(-e)[..., None] + 2.0 ** -o
    n = ((f.view(torch.int32) + ((bits << 4) | 8)) >> 20) - ((127 - o) << 3)
    if kind == "m":
        n = n.clamp(max=127)
        return torch.where(v < 0, -n, n).to(torch.int8), e.to(torch.int8)
    n = torch.where(v > 0, n.clamp(1, 254), n)
    return (n - 128).to(torch.int8), e.to(torch.int8)


def _mix(x):
    """A hash of 32-bit words, held in 64."""
    x = x ^ (x >> 16)
    x = (x * 0x7feb352d) & 0xffffffff
    x = x ^ (x >> 15)
    x = (x * 0x846ca68b) & 0xffffffff
    return x ^ (x >> 16)


def _adamw_constants(st):
    t, lr, b1, b2 = st["step"], st["lr"], st["beta1"], st["beta2"]
    return 1 - lr * st["weight_decay"], lr / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)


def _adamw_plain(case, st):
    """All tensors as one, each filled up to whole blocks of 64 as they lie in the
    buffers that hold them."""
    st["step"] += 1
    g = st["g_all"].float()
    if st["scale"] is not None:
        g = g * st["scale"]
    kept, size, root = _adamw_constants(st)
    if case["bits"] == 32:
        m, v = st["m_all"], st["v_all"]
    else:
        m, v = (_state8_values(st[k + "_all"].view(-1, BLOCK), st[k + "e_all"], k).flatten() for k in "mv")
    m = m * st["beta1"] + g * (1 - st["beta1"])
    v = v * st["beta2"] + g * (1 - st["beta2"]) * g
    p = st["p_all"] * kept - m / (torch.sqrt(v) * root + st["eps"]) * size
    st["p_all"].copy_(p)
    if case["bits"] == 32:
        st["m_all"].copy_(m)
        st["v_all"].copy_(v)
        return st["p_all"], st["m_all"], st["v_all"]
    base = _mix(torch.tensor((st["seed"] + 0x9e3779b9 * st["step"]) & 0xffffffff, device=p.device))
    keys = _mix((base + torch.arange(len(st["p"]), device=p.device)) & 0xffffffff)
    sizes = torch.tensor(st["padded"], device=p.device)
    key = keys.repeat_interleave(sizes)
    start = (sizes.cumsum(0) - sizes).repeat_interleave(sizes)
    word = _mix((torch.arange(key.numel(), device=p.device) - start) ^ key)
    for k, t, bits in (("m", m, word & 0xffff), ("v", v, word >> 16)):
        codes, exps = _state8_codes(t.view(-1, BLOCK), bits.int().view(-1, BLOCK), k)
        st[k + "_all"].copy_(codes.flatten())
        st[k + "e_all"].copy_(exps)
    return (st["p_all"], *(_state8_values(st[k + "_all"].view(-1, BLOCK), st[k + "e_all"], k).flatten() for k in "mv"))


PLAIN = {"conv_fwd": _conv_fwd, "conv_bwd": _conv_bwd, "scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd,
         "token": _token_fwd, "adamw": _adamw_plain}


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        # filled in parts: no 32-bit copy of a large 16-bit tensor is needed at once
        out = torch.empty(shape, device=dev, dtype=dtype)
        for part in out.flatten().split(1 << 26):
            part.copy_(torch.randn(part.shape, generator=g, device=dev) * std)
        return out

    st = {"case": case}
    if case["op"] == "adamw":
        return _prepare_adamw(case, st, normal, g)
    dt, B, H = DTYPES[case["dtype"]], case["B"], case["H"]
    if case["op"] in ("conv_fwd", "conv_bwd", "token"):
        W = case["W"]
        st["weight"] = normal(H, W, std=W ** -0.5)
        st["bias"] = normal(H, std=0.1)
    if "N" in case:
        N = case["N"]
        # rates 1 .. N, steps between a thousandth and a tenth at a logit of 0
        st["a_log"] = torch.log(torch.arange(1.0, N + 1, device=dev)).repeat(H, 1) + normal(H, N, std=0.1)
        step = torch.exp(torch.rand(H, generator=g, device=dev) * math.log(100) + math.log(1e-3))
        st["dt_bias"] = torch.log(torch.expm1(step))
        st["d"] = 1 + normal(H, std=0.1)
    if case["op"] == "token":
        W, slots = case["W"], 2 * B
        st["window"] = normal(slots, W - 1, H, dtype=dt)
        st["states"] = normal(slots, H, N, std=0.3)
        st["slot"] = torch.randperm(slots, generator=g, device=dev)[:B].to(torch.int32)
        st["x"], st["dt"], st["z"] = (normal(B, H, dtype=dt) for _ in range(3))
        st["xs"] = _silu(normal(B, H)).to(dt)
        st["b"], st["c"] = normal(B, N, dtype=dt), normal(B, N, dtype=dt)
        return st
    T = case["T"]
    rows = (B, T) if case["batch_first"] else (T, B)
    st["lengths"] = (torch.randint(T // 10, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
                     if case["varlen"] else None)
    st["x"] = normal(*rows, H, dtype=dt)
    if case["op"].startswith("conv"):
        st["state"] = normal(B, W - 1, H, dtype=dt)
        if case["op"] == "conv_bwd":
            st["dy"] = normal(*rows, H, dtype=dt)
        return st
    for part in st["x"].flatten().split(1 << 26):
        part.copy_(_silu(part.float()))
    st["dt"], st["z"] = (normal(*rows, H, dtype=dt) for _ in range(2))
    st["b"], st["c"] = (normal(*rows, N, dtype=dt) for _ in range(2))
    st["h0"] = normal(B, H, N, std=0.3)
    if case["op"] == "scan_bwd":
        st["states"] = _scan_fwd(dict(case, train=True), st)[2]
        st["dy"] = normal(*rows, H, dtype=dt)
        st["dh_n"] = normal(B, H, N, std=0.1)
    return st


def _prepare_adamw(case, st, normal, g):
    """Parameters, gradients and states as views of one buffer each, as a trainer lays
    them out, every tensor from a whole block of 64 on; states of a run under way."""
    shapes = _shapes(case)
    sizes = [math.prod(s) for s in shapes]
    st["padded"] = [-(-n // BLOCK) * BLOCK for n in sizes]
    total = sum(st["padded"])
    st |= {"step": 1000, "lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "seed": 7}
    st["scale"] = 0.5 + 0.5 * torch.rand(1, generator=g, device="cuda") if case["scaled"] else None
    live = torch.cat([torch.arange(p, device="cuda") < n for n, p in zip(sizes, st["padded"])])
    # gradients whose scale differs from row to row
    rms = torch.exp(normal(-(-total // 1024), std=1.5) - 5).repeat_interleave(1024)[:total]
    st["g_all"] = (normal(total) * rms * live).to(DTYPES[case["grad"]])
    st["p_all"] = normal(total, std=0.03) * live
    m, v = normal(total) * rms * 0.2 * live, (0.5 + torch.rand(total, generator=g, device="cuda")) * rms * rms * live
    if case["bits"] == 8:
        for k, t in (("m", m), ("v", v)):
            half = torch.full((1, 1), 0x7fff, dtype=torch.int32, device="cuda")
            codes, st[k + "e_all"] = _state8_codes(t.view(-1, BLOCK), half, k)
            st[k + "_all"] = codes.flatten()
    else:
        st["m_all"], st["v_all"] = m, v
    starts = [0]
    for p in st["padded"]:
        starts.append(starts[-1] + p)
    for k in ("p", "g", "m", "v"):
        st[k] = [st[k + "_all"][o:o + n].view(s) for o, n, s in zip(starts, sizes, shapes)]
        if case["bits"] == 8 and k in "mv":
            st[k] = [(t, st[k + "e_all"][o // BLOCK:(o + p) // BLOCK])
                     for t, o, p in zip(st[k], starts, st["padded"])]
    return st


# --------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if not own:
        return PLAIN[case["op"]](case, st)
    ops = _ops()
    if case["op"] == "adamw":
        st["step"] += 1
        ops.adamw_step(st["p"], st["g"], st["m"], st["v"], st["step"], lr=st["lr"],
                       betas=(st["beta1"], st["beta2"]), eps=st["eps"], weight_decay=st["weight_decay"],
                       scale=st["scale"], seed=st["seed"])
        if case["bits"] == 32:
            return st["p_all"], st["m_all"], st["v_all"]
        return (st["p_all"], ops.state8_unpack(st["m_all"], st["me_all"], signed=True),
                ops.state8_unpack(st["v_all"], st["ve_all"], signed=False))
    if case["op"] == "token":
        u = ops.conv_step(st["x"], st["weight"], st["window"], bias=st["bias"], slot=st["slot"])
        y = ops.selscan_step(st["xs"], st["dt"], st["a_log"], st["b"], st["c"], st["states"], d=st["d"],
                             dt_bias=st["dt_bias"], z=st["z"], slot=st["slot"])
        return u, st["window"], y, st["states"]
    how = {"lengths": st["lengths"], "batch_first": case["batch_first"]}
    if case["op"] == "conv_fwd":
        return ops.conv_forward(st["x"], st["weight"], bias=st["bias"], state=st["state"], **how)
    if case["op"] == "conv_bwd":
        return ops.conv_backward(st["dy"], st["x"], st["weight"], bias=st["bias"], state=st["state"], **how)
    how |= {"d": st["d"], "dt_bias": st["dt_bias"], "z": st["z"]}
    if case["op"] == "scan_fwd":
        out = ops.selscan_forward(st["x"], st["dt"], st["a_log"], st["b"], st["c"], h0=st["h0"],
                                  states=case["train"], **how)
        return list(out if case["train"] else out[:2])
    got = ops.selscan_backward(st["dy"], st["x"], st["dt"], st["a_log"], st["b"], st["c"], st["states"],
                               dh_n=st["dh_n"], **how)
    return tuple(got[k] for k in ("dx", "ddt", "db", "dc", "dz", "da_log", "dd", "ddt_bias", "dh0"))


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, st)
    f64 = torch.float64

    def sigmoid(v):
        return 0.5 * (1 + torch.tanh(0.5 * v))

    if "N" in case:
        rate, bias, skip = -torch.exp(st["a_log"].double()), st["dt_bias"].double(), st["d"].double()

    def softplus(v):
        return torch.logaddexp(v, torch.zeros_like(v))

    if case["op"] == "token":
        slot, W = st["slot"].long(), case["W"]
        window, states = st["window"].double(), st["states"].double()
        v = st["bias"].double() + st["weight"].double()[:, W - 1] * st["x"].double()
        for k in range(W - 1):
            v = v + st["weight"].double()[:, k] * window[slot, k]
        window[slot] = torch.cat([window[slot, 1:], st["x"].double()[:, None]], 1)
        x, b, c, z = (st[k].double() for k in ("xs", "b", "c", "z"))
        delta = softplus(st["dt"].double() + bias)
        h = torch.exp(delta[:, :, None] * rate) * states[slot] + torch.einsum("bh,bn->bhn", delta * x, b)
        states[slot] = h
        y = (torch.einsum("bhn,bn->bh", h, c) + skip * x) * z * sigmoid(z)
        return v * sigmoid(v), window, y, states

    T, B, H = case["T"], case["B"], case["H"]
    dev = st["x"].device

    def wide(name):
        t = st[name].double()
        return t.transpose(0, 1) if case["batch_first"] else t

    def back(t):
        return t.transpose(0, 1) if case["batch_first"] else t

    ends = torch.full((B,), T, device=dev) if st["lengths"] is None else st["lengths"]
    dead = (torch.arange(T, device=dev)[:, None] >= ends[None])[..., None]
    if case["op"].startswith("conv"):
        W, w = case["W"], st["weight"].double()
        x = torch.cat([st["state"].double().transpose(0, 1), wide("x").masked_fill(dead, 0)])
        v = torch.zeros(T, B, H, dtype=f64, device=dev) + st["bias"].double()
        for k in range(W):
            v += x[k:k + T] * w[:, k]
        s = sigmoid(v)
        if case["op"] == "conv_fwd":
            last = torch.stack([torch.stack([x[int(n) + k, row] for k in range(W - 1)])
                                for row, n in enumerate(ends.tolist())])
            return back((v * s).masked_fill(dead, 0)), last
        dv = (wide("dy") * (s + v * s * (1 - s))).masked_fill(dead, 0)
        dx = torch.zeros(T + W - 1, B, H, dtype=f64, device=dev)
        dw = torch.zeros(H, W, dtype=f64, device=dev)
        for k in range(W):
            dx[k:k + T] += dv * w[:, k]
            dw[:, k] = torch.einsum("tbh,tbh->h", dv, x[k:k + T])
        return back(dx[W - 1:].masked_fill(dead, 0)), dw, dv.sum((0, 1)), dx[:W - 1].transpose(0, 1)

    N = case["N"]
    x, b, c, z = (wide(k) for k in ("x", "b", "c", "z"))
    slope = sigmoid(wide("dt") + bias)
    delta = softplus(wide("dt") + bias).masked_fill(dead, 0)
    if case["op"] == "scan_fwd":
        h, y, states = st["h0"].double(), torch.empty_like(x), []
        for t in range(T):  # one step after another; a step past a row's end has delta 0
            if t % CHUNK == 0:
                states.append(h)
            h = torch.addcmul((delta[t] * x[t])[:, :, None] * b[t][:, None], torch.exp(delta[t][:, :, None] * rate), h)
            y[t] = (h * c[t][:, None]).sum(-1)
        y = ((y + skip * x) * z * sigmoid(z)).masked_fill(dead, 0)
        return [back(y), h] + ([torch.stack(states)] if case["train"] else [])

    dy = wide("dy").masked_fill(dead, 0)
    gate = sigmoid(z)
    gy = dy * z * gate
    before = torch.empty(T, B, H, N, dtype=f64, device=dev)
    total, dc = torch.empty_like(x), torch.empty_like(b)
    for t in range(T):
        h = st["states"][t // CHUNK].double() if t % CHUNK == 0 else h
        before[t] = h
        h = torch.addcmul((delta[t] * x[t])[:, :, None] * b[t][:, None], torch.exp(delta[t][:, :, None] * rate), h)
        total[t] = (h * c[t][:, None]).sum(-1)
        dc[t] = (gy[t][:, :, None] * h).sum(1)
    dz = dy * (total + skip * x) * (gate + z * gate * (1 - gate))
    come = st["dh_n"].double()
    dx, ddelta, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(b)
    da_log = torch.zeros(H, N, dtype=f64, device=dev)
    for t in reversed(range(T)):  # the gradient reaching each state
        e = come + gy[t][:, :, None] * c[t][:, None]
        du = (e * b[t][:, None]).sum(-1)
        come = torch.exp(delta[t][:, :, None] * rate) * e
        dlog = come * before[t] * rate
        ddelta[t] = dlog.sum(-1) + du * x[t]
        dx[t] = du * delta[t] + gy[t] * skip
        db[t] = (e * (delta[t] * x[t])[:, :, None]).sum(1)
        da_log += (dlog * delta[t][:, :, None]).sum(0)
    ddt = (ddelta * slope).masked_fill(dead, 0)
    dx = dx.masked_fill(dead, 0)
    return (*(back(v) for v in (dx, ddt, db, dc, dz)), da_log, (gy * x).sum((0, 1)), ddt.sum((0, 1)), come)


def _exact_adamw(case, st):
    t = st["step"] + 1
    g = st["g_all"].double() * (1 if st["scale"] is None else st["scale"].double())

    def state(k):
        if case["bits"] == 32:
            return st[k + "_all"].double()
        q, o = st[k + "_all"].double(), OCTAVES[k]
        n = q.abs() if k == "m" else q + 128
        # n eighths of octaves above the offset, straight lines between the octaves
        value = torch.ldexp(1 + torch.remainder(n, 8) / 8, torch.floor(n / 8) - o) - 2.0 ** -o
        value = torch.copysign(value, q) if k == "m" else value
        return torch.ldexp(value.view(-1, BLOCK), st[k + "e_all"].double()[:, None]).flatten()

    m = st["beta1"] * state("m") + (1 - st["beta1"]) * g
    v = st["beta2"] * state("v") + (1 - st["beta2"]) * g * g
    hat_m, hat_v = m / (1 - st["beta1"] ** t), v / (1 - st["beta2"] ** t)
    p = st["p_all"].double()
    p = p - st["lr"] * st["weight_decay"] * p - st["lr"] * hat_m / (hat_v.sqrt() + st["eps"])
    return (p, m, v) if case["bits"] == 32 else (p, None, None)
