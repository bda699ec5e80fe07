"""Plain 64-bit implementations of the short causal convolution, the selective
scan and the AdamW step, written step by step on the CPU; gradients are torch's of
these."""
import torch

F64 = torch.float64


def conv(x, weight, bias, silu, lengths, state):
    """y [T, B, H] and the last W - 1 inputs [B, W - 1, H]; time first, float64."""
    T, B, H = x.shape
    W = weight.shape[1]
    before = torch.zeros(B, W - 1, H, dtype=F64) if state is None else state
    rows, ends = [], []
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        seq = torch.cat([before[b], x[:n, b]])
        v = torch.zeros(n, H, dtype=F64) + (0 if bias is None else bias)
        for k in range(W):
            v = v + weight[:, k] * seq[k:k + n]
        y = v * torch.sigmoid(v) if silu else v
        rows.append(torch.cat([y, torch.zeros(T - n, H, dtype=F64)]))
        ends.append(seq[n:])
    return torch.stack(rows, 1), torch.stack(ends)


def scan(x, dt, a_log, b, c, d, dt_bias, z, lengths, h0, chunk=32, dt_in=None):
    """y [T, B, H], h_n [B, H, N] and the states before every `chunk` steps.  dt_in:
    what scales the inputs in the place of dt, which then only sets the decays."""
    T, B, H = x.shape
    N = a_log.shape[1]
    delta = dt if dt_bias is None else dt + dt_bias
    delta = torch.logaddexp(delta, torch.zeros_like(delta))
    into = delta
    if dt_in is not None:
        into = dt_in if dt_bias is None else dt_in + dt_bias
        into = torch.logaddexp(into, torch.zeros_like(into))
    h = torch.zeros(B, H, N, dtype=F64) if h0 is None else h0
    ys, states = [], []
    for t in range(T):
        if t % chunk == 0:
            states.append(h)
        on = torch.ones(B, dtype=torch.bool) if lengths is None else t < lengths
        new = torch.exp(-delta[t][..., None] * torch.exp(a_log)) * h \
            + (into[t] * x[t])[..., None] * b[t][:, None]
        h = torch.where(on[:, None, None], new, h)
        y = (new * c[t][:, None]).sum(-1)
        if d is not None:
            y = y + d * x[t]
        if z is not None:
            y = y * z[t] * torch.sigmoid(z[t])
        ys.append(torch.where(on[:, None], y, torch.zeros_like(y)))
    return torch.stack(ys), h, torch.stack(states)


def mix(x):
    m = 0xffffffff
    x ^= x >> 16
    x = x * 0x7feb352d & m
    x ^= x >> 15
    x = x * 0x846ca68b & m
    return x ^ x >> 16


def state8_value(q, e, signed):
    """What one code stands for."""
    if q == (-128 if signed else 127):
        return float("nan")
    o = 14 if signed else 30
    n = abs(q) if signed else q + 128
    f = (1 + n % 8 / 8) * 2.0 ** (n // 8 - o) - 2.0 ** -o
    return (-f if q < 0 and signed else f) * 2.0 ** e


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, scale):
    """(p, m, v) after a step, float64."""
    g = g if scale is None else g * scale
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    root = (v / (1 - betas[1] ** step)).sqrt()
    p = p * (1 - lr * weight_decay) - lr * (m / (1 - betas[0] ** step)) / (root + eps)
    return p, m, v
