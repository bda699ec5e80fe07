"""Thin ctypes binding of librcu.so (argument marshalling only).

Every function here has the name of the C entry point it calls (see
include/rcu.h) and only turns torch tensors into device pointers and CUDA
streams; every step of the computation runs in the library's kernels.  The
library must have been built (``recurrent_cell_unroll_gb300._build.build()``);
a missing library raises instead of falling back to anything else.

Inputs are re-materialised when their strides are not the C-canonical ones
(a tensor of shape [1, 4, 5] with strides (5, 5, 1) passes ``is_contiguous()``
but is not canonical; see "[Performance] LSTM/GRU scan: canonical strides +
cuDNN flat-storage clones + thread-local recurrent mode", pytorch/rl PR 3754).
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import _build

RCU_LSTM, RCU_GRU, RCU_BIDIR = 0, 1, 0x100
RCU_F32, RCU_BF16, RCU_I8 = 0, 1, 2
RCU_OK, RCU_ERR_INVALID, RCU_ERR_UNSUPPORTED, RCU_ERR_CUDA = 0, -1, -2, -3
RCU_ERR_TIMEOUT, RCU_ERR_LENGTHS, RCU_ERR_STATE, RCU_ERR_SLOTS = -4, -5, -6, -7
RCU_ATTR_BARRIER_TIMEOUT_NS, RCU_ATTR_TEST_DROP_ARRIVAL, RCU_ATTR_FORCE_PATH = 1, 2, 3
RCU_ATTR_PROFILE, RCU_ATTR_TRACE, RCU_ATTR_TC_KSPLIT = 4, 5, 7
RCU_ATTR_LAYER_PIPELINE = 10
RCU_CLIP_CELL, RCU_CLIP_PROJ = 0, 1
RCU_ATTR_HOST_CHUNKS, RCU_MAX_HOST_CHUNKS = 8, 16
RCU_TIME_FIRST, RCU_BATCH_FIRST = 0, 1
RCU_LINREC_CHUNK, RCU_ACT8_BLOCK = 64, 64

EXPORTED = (
    "rcu_last_error", "rcu_version", "rnn_create", "rnn_set_weights", "rnn_forward",
    "rnn_get_pack", "rnn_get_status", "rnn_set_attr", "rnn_set_clip", "rnn_last_launch_count",
    "rnn_destroy",
    "rnn_profile_entry", "rnn_profile_reset", "rnn_get_trace", "rnn_lstm_forward_noalloc",
    "rssm_create", "rssm_set_weights", "rssm_unroll", "rssm_get_status",
    "rssm_last_launch_count", "rssm_destroy", "rssm_set_attr", "rssm_get_trace",
    "rssm_set_actor", "rssm_unroll_actor", "rnn_forward_host", "rssm_unroll_host",
    "rssm_unroll_actor_host", "rnn_backward", "rnn_get_weight_grads", "rssm_backward",
    "rssm_get_weight_grads", "rssm_profile_entry", "rssm_profile_reset", "rssm_backward_actor",
    "rssm_get_actor_grads", "rnn_host_plan",
    "rcu_seq_create", "rcu_seq_destroy", "rcu_seq_get_status", "rcu_seq_set_attr",
    "rcu_seq_profile_entry", "rcu_seq_profile_reset", "rcu_seq_last_launch_count",
    "rcu_linrec_forward", "rcu_linrec_backward", "rcu_linrec_step", "rcu_layernorm_forward",
    "rcu_layernorm_backward", "rcu_act8_pack", "rcu_act8_unpack",
)

_lib = None
_lock = threading.Lock()


class RcuError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"rcu error {code}: {msg}")
        self.code = code


def lib_path() -> str:
    return _build.LIB


def signatures() -> dict:
    """ctypes (restype, argtypes) of every entry point of include/rcu.h."""
    P, I, I64, D = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double
    return {
        "rcu_last_error": (ctypes.c_char_p, []),
        "rcu_version": (ctypes.c_char_p, []),
        "rnn_create": (I, [ctypes.POINTER(P), I, I, I, I, I, I]),
        "rnn_set_weights": (I, [P, I, I, P, P, P, P, P, P]),
        "rnn_forward": (I, [P, I, I, P, P, P, P, P, P, P, P, P]),
        "rnn_get_pack": (I, [P, P, P, P, P]),
        "rnn_get_status": (I, [P, P]),
        "rnn_set_attr": (I, [P, I, I64]),
        "rnn_set_clip": (I, [P, I, I, ctypes.c_double, ctypes.c_double]),
        "rnn_last_launch_count": (I, [P]),
        "rnn_host_plan": (I, [P, ctypes.POINTER(I), ctypes.POINTER(I), ctypes.POINTER(I)]),
        "rnn_destroy": (I, [P]),
        "rnn_profile_entry": (I, [P, I, ctypes.POINTER(ctypes.c_char_p),
                                  ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I64)]),
        "rnn_profile_reset": (I, [P]),
        "rnn_get_trace": (I, [P, P, I, P]),
        "rnn_lstm_forward_noalloc": (I, [I, I, I, I] + [P] * 10 + [P]),
        "rssm_create": (I, [ctypes.POINTER(P), I, I, I, I]),
        "rssm_set_weights": (I, [P] + [P] * 10 + [P]),
        "rssm_unroll": (I, [P, I, I] + [P] * 8 + [P]),
        "rssm_get_status": (I, [P, P]),
        "rssm_last_launch_count": (I, [P]),
        "rssm_destroy": (I, [P]),
        "rssm_set_attr": (I, [P, I, I64]),
        "rssm_get_trace": (I, [P, P, I, P]),
        "rssm_set_actor": (I, [P, I, P, P, P, P, P]),
        "rssm_unroll_actor": (I, [P, I, I] + [P] * 8 + [P]),
        "rnn_forward_host": (I, [P, I, I] + [P] * 8),
        "rnn_backward": (I, [P, I, I] + [P] * 11),
        "rnn_get_weight_grads": (I, [P, I, I, P, P, P, P, P, P]),
        "rssm_unroll_host": (I, [P, I, I] + [P] * 8 + [P]),
        "rssm_unroll_actor_host": (I, [P, I, I] + [P] * 8 + [P]),
        "rssm_backward": (I, [P, I, I] + [P] * 12),
        "rssm_get_weight_grads": (I, [P] + [P] * 11),
        "rssm_backward_actor": (I, [P, I, I] + [P] * 11),
        "rssm_get_actor_grads": (I, [P] * 6),
        "rssm_profile_entry": (I, [P, I, ctypes.POINTER(ctypes.c_char_p),
                                   ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I64)]),
        "rssm_profile_reset": (I, [P]),
        "rcu_seq_create": (I, [ctypes.POINTER(P)]),
        "rcu_seq_destroy": (I, [P]),
        "rcu_seq_get_status": (I, [P, P]),
        "rcu_seq_set_attr": (I, [P, I, I64]),
        "rcu_seq_profile_entry": (I, [P, I, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(D),
                                      ctypes.POINTER(I64)]),
        "rcu_seq_profile_reset": (I, [P]),
        "rcu_seq_last_launch_count": (I, [P]),
        "rcu_linrec_forward": (I, [P, I, I, I, I, I] + [P, I64] * 3 + [P, D, P, P, P, I64, P, P,
                                                                       P]),
        "rcu_linrec_backward": (I, [P, I, I, I, I, I, I] + [P, I64] * 3 + [P, P, P, P, D, P, P]
                                + [P, I64, P] + [P, I64] * 3 + [P, P, P]),
        "rcu_linrec_step": (I, [P, I, I, I] + [P, I64] * 3 + [P, D, P, I, P, P, I64, P]),
        "rcu_layernorm_forward": (I, [P, I, I64, I, P, I64, P, I64, P, P, D, P, I64, P, I64, P, P,
                                      P]),
        "rcu_layernorm_backward": (I, [P, I, I, I64, I, P, I64, P, I64, P, P, P, P, P, I64, P, I64,
                                       P, P, P]),
        "rcu_act8_pack": (I, [P, I, I64, I, P, I64, P, I64, P, P]),
        "rcu_act8_unpack": (I, [P, I, I64, I, P, I64, P, P, I64, P]),
    }


def load(path: Optional[str] = None):
    """Load librcu.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _build.LIB
        if not os.path.exists(p):
            raise RuntimeError(f"librcu.so not found at {p}: build it with "
                               "recurrent_cell_unroll_gb300._build.build()")
        lib = ctypes.CDLL(p)
        sig = signatures()
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(rc: int) -> int:
    if rc != RCU_OK:
        raise RcuError(rc, load().rcu_last_error().decode())
    return rc


def canonical_contiguous(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """Return t if its strides are the C-canonical ones, else a canonical copy."""
    if t is None:
        return None
    expect, acc = [], 1
    for n in reversed(t.shape):
        expect.append(acc)
        acc *= n
    if tuple(reversed(expect)) == tuple(t.stride()) and t.storage_offset() >= 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _dev(t: Optional[torch.Tensor], dtype=torch.float32):
    if t is None:
        return None, None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if t.dtype != dtype:
        raise ValueError(f"expected {dtype}, got {t.dtype}")
    t = canonical_contiguous(t)
    return t, ctypes.c_void_p(t.data_ptr())


def _host(t: Optional[torch.Tensor], dtype=torch.float32, out=False):
    """Host tensor -> (kept tensor, pointer).  Pinned tensors (pin_memory) are
    used in place by the kernels; pageable ones are staged by the library."""
    if t is None:
        return None, None
    if t.is_cuda:
        raise ValueError("the *_host entry points take host tensors")
    if t.dtype != dtype:
        raise ValueError(f"expected {dtype}, got {t.dtype}")
    if out:
        if canonical_contiguous(t) is not t:
            raise ValueError("outputs must be C-contiguous")
    else:
        t = canonical_contiguous(t)
    return t, ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


# --------------------------------------------------------------------------- C names

def rcu_version() -> str:
    return load().rcu_version().decode()


def rnn_create(cell: int, layers: int, in_dim: int, hidden: int, proj: int = 0,
               dtype: int = RCU_F32) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load().rnn_create(ctypes.byref(h), cell, layers, in_dim, hidden, proj, dtype))
    return h


def rnn_set_weights(h, layer: int, direction: int, W_ih, W_hh, b_ih=None, b_hh=None, W_hr=None,
                    stream=None):
    keep = [_dev(t) for t in (W_ih, W_hh, b_ih, b_hh, W_hr)]
    _check(load().rnn_set_weights(h, layer, direction, *[k[1] for k in keep], _stream(stream)))


def rnn_forward(h, T: int, B: int, x, lengths, h0, c0, eps, y, h_n, c_n, stream=None):
    x_, xp = _dev(x)
    l_, lp = _dev(lengths, torch.int32)
    h0_, h0p = _dev(h0)
    c0_, c0p = _dev(c0)
    e_, ep = _dev(eps)
    for out in (y, h_n, c_n):
        if out is not None and not out.is_contiguous():
            raise ValueError("outputs must be contiguous")
    _, yp = _dev(y)
    _, hnp = _dev(h_n)
    _, cnp = _dev(c_n)
    _check(load().rnn_forward(h, T, B, xp, lp, h0p, c0p, ep, yp, hnp, cnp, _stream(stream)))


def rnn_get_pack(h, sorted_idx, unsorted_idx, batch_sizes, stream=None):
    _check(load().rnn_get_pack(h, *[_dev(t, torch.int32)[1] for t in
                                   (sorted_idx, unsorted_idx, batch_sizes)], _stream(stream)))


def rnn_get_status(h, stream=None) -> int:
    """Synchronise and return the device status code (0 = ok); does not raise."""
    return load().rnn_get_status(h, _stream(stream))


def rnn_set_attr(h, attr: int, value: int):
    _check(load().rnn_set_attr(h, attr, value))


def rnn_last_launch_count(h) -> int:
    return load().rnn_last_launch_count(h)


def rnn_profile_entry(h, i: int):
    """(name, total_ms, launches) of profile entry i, or None past the end."""
    name, ms, n = ctypes.c_char_p(), ctypes.c_double(), ctypes.c_int64()
    rc = load().rnn_profile_entry(h, i, ctypes.byref(name), ctypes.byref(ms), ctypes.byref(n))
    if rc != RCU_OK:
        return None
    return name.value.decode(), ms.value, n.value


def rnn_profile_reset(h):
    _check(load().rnn_profile_reset(h))


def rssm_profile_entry(h, i: int):
    """(name, total_ms, count) of RSSM profile entry i, or None past the end."""
    name, ms, n = ctypes.c_char_p(), ctypes.c_double(), ctypes.c_int64()
    rc = load().rssm_profile_entry(h, i, ctypes.byref(name), ctypes.byref(ms), ctypes.byref(n))
    if rc != RCU_OK:
        return None
    return name.value.decode(), ms.value, n.value


def rssm_profile_reset(h):
    _check(load().rssm_profile_reset(h))


def rnn_get_trace(h, n_steps: int, stream=None):
    """[n_steps, 16] int64 global-timer stamps of the first layer (see rcu.h)."""
    out = torch.zeros((n_steps, 16), dtype=torch.int64)
    _check(load().rnn_get_trace(h, ctypes.c_void_p(out.data_ptr()), n_steps, _stream(stream)))
    return out


def rnn_destroy(h):
    if h:
        load().rnn_destroy(h)


def rnn_lstm_forward_noalloc(T: int, B: int, in_dim: int, hidden: int, x, W_ih, W_hh,
                             b_ih=None, b_hh=None, h0=None, c0=None, y=None, h_n=None, c_n=None,
                             stream=None):
    """One-layer fp32 LSTM through the allocation-free entry point (see rcu.h)."""
    ins = [_dev(t) for t in (x, W_ih, W_hh, b_ih, b_hh, h0, c0)]
    outs = [_dev(t) for t in (y, h_n, c_n)]
    _check(load().rnn_lstm_forward_noalloc(T, B, in_dim, hidden, *[k[1] for k in ins],
                                           *[k[1] for k in outs], _stream(stream)))


def rnn_forward_host(h, T: int, B: int, x, lengths, h0, c0, y, h_n, c_n, stream=None):
    """rnn_forward on host tensors (see rcu.h); results are in y/h_n/c_n once
    the stream has passed the call."""
    ins = [_host(x), _host(lengths, torch.int32), _host(h0), _host(c0)]
    outs = [_host(t, out=True) for t in (y, h_n, c_n)]
    _check(load().rnn_forward_host(h, T, B, *[k[1] for k in ins], *[k[1] for k in outs],
                                   _stream(stream)))


def rnn_host_plan(h) -> dict:
    """How the last rnn_forward_host call moved x and y (see rcu.h)."""
    c, xi, yi = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(load().rnn_host_plan(h, ctypes.byref(c), ctypes.byref(xi), ctypes.byref(yi)))
    return {"chunks": c.value, "x_in_place": bool(xi.value), "y_in_place": bool(yi.value)}


def rnn_backward(h, T: int, B: int, x, lengths, h0, c0, dy, dh_n, dc_n, dx, dh0, dc0,
                 stream=None):
    """Backward pass through time (see rcu.h); device tensors."""
    ins = [_dev(x), _dev(lengths, torch.int32)] + [_dev(t) for t in (h0, c0, dy, dh_n, dc_n)]
    outs = [_dev(t) for t in (dx, dh0, dc0)]
    _check(load().rnn_backward(h, T, B, *[k[1] for k in ins], *[k[1] for k in outs],
                               _stream(stream)))


def rnn_get_weight_grads(h, layer: int, dW_ih, dW_hh, db_ih, db_hh, dW_hr=None, stream=None,
                         direction: int = 0):
    outs = [_dev(t) for t in (dW_ih, dW_hh, db_ih, db_hh, dW_hr)]
    _check(load().rnn_get_weight_grads(h, layer, direction, *[k[1] for k in outs],
                                       _stream(stream)))


def rssm_create(state_dim: int, action_dim: int, hidden: int, rnn_hidden: int):
    h = ctypes.c_void_p()
    _check(load().rssm_create(ctypes.byref(h), state_dim, action_dim, hidden, rnn_hidden))
    return h


def rssm_set_weights(h, W1, b1, W_ih, W_hh, b_ih, b_hh, W2, b2, W3, b3, stream=None):
    keep = [_dev(t) for t in (W1, b1, W_ih, W_hh, b_ih, b_hh, W2, b2, W3, b3)]
    _check(load().rssm_set_weights(h, *[k[1] for k in keep], _stream(stream)))


def rssm_unroll(h, T: int, B: int, state0, belief0, actions, eps, means, stds, states, beliefs,
                stream=None):
    ins = [_dev(t) for t in (state0, belief0, actions, eps)]
    outs = [_dev(t) for t in (means, stds, states, beliefs)]
    _check(load().rssm_unroll(h, T, B, *[k[1] for k in ins], *[k[1] for k in outs],
                              _stream(stream)))


def rssm_backward(h, T: int, B: int, state0, belief0, actions, eps, dmeans, dstds, dstates,
                  dbeliefs, dstate0, dbelief0, dactions, stream=None):
    """Backward pass through time of rssm_unroll (see rcu.h); device tensors."""
    ins = [_dev(t) for t in (state0, belief0, actions, eps, dmeans, dstds, dstates, dbeliefs)]
    outs = [_dev(t) for t in (dstate0, dbelief0, dactions)]
    _check(load().rssm_backward(h, T, B, *[k[1] for k in ins], *[k[1] for k in outs],
                                _stream(stream)))


def rssm_backward_actor(h, T: int, B: int, state0, belief0, eps, dmeans, dstds, dstates,
                        dbeliefs, dstate0, dbelief0, dactions, stream=None):
    """Backward pass through time of rssm_unroll_actor (see rcu.h); device tensors."""
    ins = [_dev(t) for t in (state0, belief0, eps, dmeans, dstds, dstates, dbeliefs)]
    outs = [_dev(t) for t in (dstate0, dbelief0, dactions)]
    _check(load().rssm_backward_actor(h, T, B, *[k[1] for k in ins], *[k[1] for k in outs],
                                      _stream(stream)))


RSSM_ACTOR_NAMES = ("Wa1", "ba1", "Wa2", "ba2")


def rssm_get_actor_grads(h, grads: dict, stream=None):
    """Copy the last rssm_backward_actor's actor gradients into the device
    tensors of grads (keys of RSSM_ACTOR_NAMES; missing or None are skipped)."""
    outs = [_dev(grads.get(k)) for k in RSSM_ACTOR_NAMES]
    _check(load().rssm_get_actor_grads(h, *[k[1] for k in outs], _stream(stream)))


RSSM_WEIGHT_NAMES = ("W1", "b1", "W_ih", "W_hh", "b_ih", "b_hh", "W2", "b2", "W3", "b3")


def rssm_weight_shapes(S: int, A: int, Hd: int, RH: int) -> dict:
    """Shapes of the prior's weights (rssm_set_weights' layouts) by name."""
    return {"W1": (Hd, S + A), "b1": (Hd,), "W_ih": (3 * RH, Hd), "W_hh": (3 * RH, RH),
            "b_ih": (3 * RH,), "b_hh": (3 * RH,), "W2": (Hd, RH), "b2": (Hd,),
            "W3": (2 * S, Hd), "b3": (2 * S,)}


def rssm_get_weight_grads(h, grads: dict, stream=None):
    """Copy the last rssm_backward's weight gradients into the device tensors
    of grads (keys of RSSM_WEIGHT_NAMES; missing or None are skipped)."""
    outs = [_dev(grads.get(k)) for k in RSSM_WEIGHT_NAMES]
    _check(load().rssm_get_weight_grads(h, *[k[1] for k in outs], _stream(stream)))


def rssm_set_actor(h, actor_hidden: int, Wa1, ba1, Wa2, ba2, stream=None):
    keep = [_dev(t) for t in (Wa1, ba1, Wa2, ba2)]
    _check(load().rssm_set_actor(h, actor_hidden, *[k[1] for k in keep], _stream(stream)))


def rssm_unroll_actor(h, T: int, B: int, state0, belief0, eps, means, stds, states, beliefs,
                      actions_out, stream=None):
    ins = [_dev(t) for t in (state0, belief0, eps)]
    outs = [_dev(t) for t in (means, stds, states, beliefs, actions_out)]
    _check(load().rssm_unroll_actor(h, T, B, *[k[1] for k in ins], *[k[1] for k in outs],
                                    _stream(stream)))


def rssm_unroll_host(h, T: int, B: int, state0, belief0, actions, eps, means, stds, states,
                     beliefs, stream=None):
    ins = [_host(t) for t in (state0, belief0, actions, eps)]
    outs = [_host(t, out=True) for t in (means, stds, states, beliefs)]
    _check(load().rssm_unroll_host(h, T, B, *[k[1] for k in ins], *[k[1] for k in outs],
                                   _stream(stream)))


def rssm_unroll_actor_host(h, T: int, B: int, state0, belief0, eps, means, stds, states, beliefs,
                           actions_out, stream=None):
    ins = [_host(t) for t in (state0, belief0, eps)]
    outs = [_host(t, out=True) for t in (means, stds, states, beliefs, actions_out)]
    _check(load().rssm_unroll_actor_host(h, T, B, *[k[1] for k in ins],
                                         *[k[1] for k in outs], _stream(stream)))


def rssm_get_status(h, stream=None) -> int:
    return load().rssm_get_status(h, _stream(stream))


def rssm_last_launch_count(h) -> int:
    return load().rssm_last_launch_count(h)


def rssm_set_attr(h, attr: int, value: int):
    _check(load().rssm_set_attr(h, attr, value))


def rssm_get_trace(h, n_steps: int, stream=None):
    """[n_steps, 16] int64 stamps of the last traced rssm_unroll (see rcu.h)."""
    out = torch.zeros((n_steps, 16), dtype=torch.int64)
    _check(load().rssm_get_trace(h, ctypes.c_void_p(out.data_ptr()), n_steps, _stream(stream)))
    return out


def rssm_destroy(h):
    if h:
        load().rssm_destroy(h)


# --------------------------------------------------------------------------- convenience wrappers

class RNN:
    """Owns an rnn handle; weights from the seeded-workload dict layout."""

    def __init__(self, cell: str, layers: int, in_dim: int, hidden: int, proj: int = 0,
                 bidirectional: bool = False, dtype: str = "f32"):
        c = RCU_LSTM if cell == "lstm" else RCU_GRU
        if bidirectional:
            c |= RCU_BIDIR
        self.cell, self.layers, self.hidden, self.proj = cell, layers, hidden, proj
        self.in_dim = in_dim
        self.D = 2 if bidirectional else 1
        self.Hout = proj if proj > 0 else hidden
        self.h = rnn_create(c, layers, in_dim, hidden, proj, RCU_BF16 if dtype == "bf16" else RCU_F32)

    @classmethod
    def from_spec(cls, spec):
        return cls(spec.cell, spec.layers, spec.in_dim, spec.hidden, spec.proj, spec.bidir, spec.dtype)

    def set_weights(self, weights, device="cuda", stream=None):
        for i, w in enumerate(weights):
            layer, d = divmod(i, self.D)
            t = {k: (None if v is None else v.to(device=device, dtype=torch.float32))
                 for k, v in w.items()}
            rnn_set_weights(self.h, layer, d, t["w_ih"], t["w_hh"], t.get("b_ih"), t.get("b_hh"),
                            t.get("w_hr"), stream)

    def _shapes(self, x, lengths=None, h0=None, c0=None, **seq):
        """The C ABI takes plain pointers and reads every tensor at the size
        the handle and (T, B) imply: a tensor of another shape is an error
        here, before any pointer crosses."""
        if x.dim() != 3 or x.shape[2] != self.in_dim:
            raise ValueError(f"x must be [T, B, {self.in_dim}], got {tuple(x.shape)}")
        T, B, _ = x.shape
        LD = self.layers * self.D
        want = {"lengths": (B,), "h0": (LD, B, self.Hout), "c0": (LD, B, self.hidden)}
        want.update({k: (T, B, self.D * self.Hout) if k in ("dy", "out") else
                     (LD, B, self.Hout if k == "dh_n" else self.hidden) for k in seq})
        for k, t in dict(lengths=lengths, h0=h0, c0=c0, **seq).items():
            if t is not None and tuple(t.shape) != want[k]:
                raise ValueError(f"{k} must be {list(want[k])}, got {list(t.shape)}")
        return T, B

    def forward(self, x, lengths=None, h0=None, c0=None, out=None, stream=None):
        T, B = self._shapes(x, lengths, h0, c0, out=out)
        dev = x.device
        y = out if out is not None else torch.empty((T, B, self.D * self.Hout), device=dev)
        hn = torch.empty((self.layers * self.D, B, self.Hout), device=dev)
        cn = torch.empty((self.layers * self.D, B, self.hidden), device=dev) \
            if self.cell == "lstm" else None
        rnn_forward(self.h, T, B, x, lengths, h0, c0, None, y, hn, cn, stream)
        return y, hn, cn

    def backward(self, x, dy, lengths=None, h0=None, c0=None, dh_n=None, dc_n=None, stream=None):
        """Gradients of a loss with dL/dy = dy (and dL/dh_n, dL/dc_n) through
        the forward on x (with lengths: int32 [B] on the device): returns (dx, dh0, dc0 or None, weight grads as a
        list over layers of dicts w_ih, w_hh, b_ih, b_hh)."""
        T, B = self._shapes(x, lengths, h0, c0, dy=dy, dh_n=dh_n, dc_n=dc_n)
        in_dim = x.shape[2]
        dev = x.device
        dx = torch.empty_like(x)
        LD = self.layers * self.D
        dh0 = torch.empty((LD, B, self.Hout), device=dev)
        dc0 = torch.empty((LD, B, self.hidden), device=dev) if self.cell == "lstm" else None
        rnn_backward(self.h, T, B, x, lengths, h0, c0, dy, dh_n, dc_n, dx, dh0, dc0, stream)
        nG = 4 if self.cell == "lstm" else 3
        grads = []  # over layer * D + direction, like the weights
        for i in range(LD):
            layer, d = divmod(i, self.D)
            k = in_dim if layer == 0 else self.D * self.Hout
            g = {"w_ih": torch.empty((nG * self.hidden, k), device=dev),
                 "w_hh": torch.empty((nG * self.hidden, self.Hout), device=dev),
                 "b_ih": torch.empty((nG * self.hidden,), device=dev),
                 "b_hh": torch.empty((nG * self.hidden,), device=dev),
                 "w_hr": torch.empty((self.proj, self.hidden), device=dev) if self.proj else None}
            rnn_get_weight_grads(self.h, layer, g["w_ih"], g["w_hh"], g["b_ih"], g["b_hh"],
                                 g["w_hr"], stream, direction=d)
            grads.append(g)
        return dx, dh0, dc0, grads

    def status(self, stream=None) -> int:
        return rnn_get_status(self.h, stream)

    def set_attr(self, attr, value):
        rnn_set_attr(self.h, attr, value)

    def set_clip(self, what: int, bounds=None):
        """Clamp the LSTM cell state (RCU_CLIP_CELL) or the projected hidden
        state (RCU_CLIP_PROJ) to bounds = (lo, hi); None turns it off."""
        if bounds is None:
            _check(load().rnn_set_clip(self.h, what, 0, 0.0, 0.0))
        else:
            _check(load().rnn_set_clip(self.h, what, 1, float(bounds[0]), float(bounds[1])))

    def launch_count(self) -> int:
        return rnn_last_launch_count(self.h)

    def profile(self) -> dict:
        """{kernel name: (total_ms, launches)} recorded while RCU_ATTR_PROFILE is on."""
        out, i = {}, 0
        while True:
            e = rnn_profile_entry(self.h, i)
            if e is None:
                return out
            out[e[0]] = (e[1], e[2])
            i += 1

    def close(self):
        if self.h:
            rnn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class RSSM:
    """Owns an rssm handle."""

    def __init__(self, state_dim: int, action_dim: int, hidden: int, rnn_hidden: int):
        self.S, self.A, self.Hd, self.RH = state_dim, action_dim, hidden, rnn_hidden
        self.Ha = 0  # actor width once set_actor has run
        self.h = rssm_create(state_dim, action_dim, hidden, rnn_hidden)

    def set_weights(self, w, device="cuda", stream=None):
        t = {k: (None if v is None else v.to(device=device, dtype=torch.float32))
             for k, v in w.items()}
        rssm_set_weights(self.h, t["W1"], t.get("b1"), t["W_ih"], t["W_hh"], t.get("b_ih"),
                         t.get("b_hh"), t["W2"], t.get("b2"), t["W3"], t.get("b3"), stream)

    def unroll(self, actions, eps, state0=None, belief0=None, stream=None):
        T, B, _ = eps.shape
        dev = eps.device
        means = torch.empty((T, B, self.S), device=dev)
        stds = torch.empty_like(means)
        states = torch.empty_like(means)
        beliefs = torch.empty((T, B, self.RH), device=dev)
        rssm_unroll(self.h, T, B, state0, belief0, actions, eps, means, stds, states, beliefs,
                    stream)
        return means, stds, states, beliefs

    def backward(self, actions, eps, state0=None, belief0=None, dmeans=None, dstds=None,
                 dstates=None, dbeliefs=None, stream=None):
        """Gradients of a loss with the given gradients with respect to the
        unroll's outputs (None = 0): returns (dstate0, dbelief0, dactions,
        dict of weight gradients keyed like set_weights)."""
        T, B, _ = eps.shape
        dev = eps.device
        dstate0 = torch.empty((B, self.S), device=dev)
        dbelief0 = torch.empty((B, self.RH), device=dev)
        dactions = torch.empty((T, B, self.A), device=dev) if self.A > 0 else None
        rssm_backward(self.h, T, B, state0, belief0, actions, eps, dmeans, dstds, dstates,
                      dbeliefs, dstate0, dbelief0, dactions, stream)
        S, A, Hd, RH = self.S, self.A, self.Hd, self.RH
        shapes = rssm_weight_shapes(S, A, Hd, RH)
        grads = {k: torch.empty(shapes[k], device=dev) for k in RSSM_WEIGHT_NAMES}
        rssm_get_weight_grads(self.h, grads, stream)
        return dstate0, dbelief0, dactions, grads

    def backward_actor(self, eps, state0=None, belief0=None, dmeans=None, dstds=None,
                       dstates=None, dbeliefs=None, stream=None):
        """Backward pass of unroll_actor: returns (dstate0, dbelief0, dactions
        (the gradient reaching each produced action), dict of the prior's
        weight gradients, dict of the actor's: Wa1, ba1, Wa2, ba2)."""
        T, B, _ = eps.shape
        dev = eps.device
        dstate0 = torch.empty((B, self.S), device=dev)
        dbelief0 = torch.empty((B, self.RH), device=dev)
        dactions = torch.empty((T, B, self.A), device=dev)
        rssm_backward_actor(self.h, T, B, state0, belief0, eps, dmeans, dstds, dstates, dbeliefs,
                            dstate0, dbelief0, dactions, stream)
        S, A, Hd, RH, Ha = self.S, self.A, self.Hd, self.RH, self.Ha
        shapes = rssm_weight_shapes(S, A, Hd, RH)
        grads = {k: torch.empty(shapes[k], device=dev) for k in RSSM_WEIGHT_NAMES}
        rssm_get_weight_grads(self.h, grads, stream)
        ashapes = {"Wa1": (Ha, S + RH), "ba1": (Ha,), "Wa2": (A, Ha), "ba2": (A,)}
        agrads = {k: torch.empty(ashapes[k], device=dev) for k in RSSM_ACTOR_NAMES}
        rssm_get_actor_grads(self.h, agrads, stream)
        return dstate0, dbelief0, dactions, grads, agrads

    def set_actor(self, a, device="cuda", stream=None):
        """Actor of the second unroll variant: dict Wa1 [Ha, S+RH], ba1 [Ha],
        Wa2 [A, Ha], ba2 [A] (biases may be None)."""
        t = {k: (None if v is None else v.to(device=device, dtype=torch.float32))
             for k, v in a.items()}
        rssm_set_actor(self.h, t["Wa1"].shape[0], t["Wa1"], t.get("ba1"), t["Wa2"],
                       t.get("ba2"), stream)
        self.Ha = t["Wa1"].shape[0]

    def unroll_actor(self, eps, state0=None, belief0=None, stream=None):
        """Unroll over eps' T steps with the actions computed by the actor;
        returns (means, stds, states, beliefs, actions)."""
        T, B, _ = eps.shape
        dev = eps.device
        means = torch.empty((T, B, self.S), device=dev)
        stds = torch.empty_like(means)
        states = torch.empty_like(means)
        beliefs = torch.empty((T, B, self.RH), device=dev)
        actions = torch.empty((T, B, self.A), device=dev)
        rssm_unroll_actor(self.h, T, B, state0, belief0, eps, means, stds, states, beliefs,
                          actions, stream)
        return means, stds, states, beliefs, actions

    def launch_count(self) -> int:
        return rssm_last_launch_count(self.h)

    def set_attr(self, attr, value):
        rssm_set_attr(self.h, attr, value)

    def profile(self) -> dict:
        """{phase name: (total_ms, count)} recorded while RCU_ATTR_PROFILE is on."""
        out, i = {}, 0
        while True:
            e = rssm_profile_entry(self.h, i)
            if e is None:
                return out
            out[e[0]] = (e[1], e[2])
            i += 1

    def close(self):
        if self.h:
            rssm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SeqOps:
    """The sequence operators (gated linear recurrence, layer norm, 8-bit
    activation checkpoints; see rcu.h) on torch tensors of the device that was
    current when it was made.

    Matrices are float32 or bfloat16.  A tensor whose rows are dense and evenly
    spaced (a slice of a wider tensor's last dimension) is used in place, one
    of any other layout as a contiguous copy.  Parameters, states and
    statistics are float32.  With ``stream`` the outputs are allocated for
    that stream, and work on it follows what it held before: a caller that
    made an input on another stream orders the two, and keeps the input until
    the work is done (``Tensor.record_stream``).  One stream at a time uses a
    SeqOps: its calls share a workspace, so calls that overlap on the GPU, on
    two streams or in a replayed graph beside them, need one each.
    """

    _DTYPES = {torch.float32: RCU_F32, torch.bfloat16: RCU_BF16}

    def __init__(self):
        self.h = None
        h = ctypes.c_void_p()
        self.lib = load()
        self.device = torch.cuda.current_device()
        _check(self.lib.rcu_seq_create(ctypes.byref(h)))
        self.h = h

    # ---- arguments
    #
    # A call on small tensors is bound by this marshalling, so each operand takes
    # one pass of cheap checks; what does not pass them goes to _refuse_or_copy.
    # A copy stays alive in `keep` until the call is enqueued (its memory is then
    # reused in stream order).

    def _refuse_or_copy(self, t, name, dtype, shape, keep):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a tensor on a CUDA device")
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the handle on "
                             f"cuda:{self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        t = t.clone(memory_format=torch.contiguous_format)
        keep.append(t)
        return t

    def _dense(self, t, name, dtype, shape, keep):
        """Pointer of a dense operand; None stays NULL."""
        if t is None:
            return None
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                and t.get_device() == self.device and t.is_contiguous()):
            t = self._refuse_or_copy(t, name, dtype, shape, keep)
        return t.data_ptr()

    def _rows(self, t, name, dtype, shape, keep):
        """(pointer, row stride) of a matrix operand: in place where its rows
        are dense and evenly spaced."""
        if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                and t.get_device() == self.device):
            if t.is_contiguous():
                return t.data_ptr(), shape[-1]
            st = t.stride()
            if len(st) > 1 and st[-1] == 1 and st[-2] >= shape[-1] and all(
                    st[k] == st[k + 1] * shape[k + 1] for k in range(len(st) - 2)):
                return t.data_ptr(), st[-2]
        return self._refuse_or_copy(t, name, dtype, shape, keep).data_ptr(), shape[-1]

    def _saved(self, t, name, dtype, shape, keep):
        """(pointer, row stride, exponents' pointer) of a backward's saved
        input: a tensor, or an 8-bit checkpoint (codes, exponents)."""
        if isinstance(t, torch.Tensor):
            return (*self._rows(t, name, dtype, shape, keep), None)
        codes, exps = t
        return (*self._rows(codes, name + "'s codes", torch.int8, shape, keep),
                self._dense(exps, name + "'s exponents", torch.int8,
                            (*shape[:-1], -(-shape[-1] // RCU_ACT8_BLOCK)), keep))

    def _type(self, t, name, dims=None):
        """(torch dtype, RCU_* type, shape) of the operand that sets them."""
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor on a CUDA device")
        shape = t.shape
        dt = self._DTYPES.get(t.dtype)
        if dt is None:
            raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
        if len(shape) != dims if dims else len(shape) < 1:
            raise ValueError(f"{name} must have {dims or 'at least one'} dimensions, "
                             f"got {list(shape)}")
        return t.dtype, dt, shape

    def _on_stream(self, stream, call, *args):
        """The call with `stream` as the current stream, so that what it
        allocates belongs to it."""
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device)
        with torch.cuda.stream(stream):
            return call(*args)

    def _raw_stream(self):
        return torch._C._cuda_getCurrentRawStream(self.device)

    # ---- gated linear recurrence

    def linrec_forward(self, x, r, i, lam, c=8.0, lengths=None, h0=None, batch_first=False,
                       states=False, stream=None):
        """y, h_n and, with states=True, what linrec_backward needs (else
        None).  x, r, i: [T, B, H] (batch_first: [B, T, H]); lam [H]; lengths
        int32 [B]; h0 [B, H]."""
        if stream is not None:
            return self._on_stream(stream, self.linrec_forward, x, r, i, lam, c, lengths, h0,
                                   batch_first, states)
        dtype, dt, shape = self._type(x, "x", 3)
        T, B, H = shape
        if batch_first:
            T, B = B, T
        keep, f32, dev = [], torch.float32, x.device
        xp, xl = self._rows(x, "x", dtype, shape, keep)
        rp, rl = self._rows(r, "r", dtype, shape, keep)
        ip, il = self._rows(i, "i", dtype, shape, keep)
        lp = self._dense(lam, "lam", f32, (H,), keep)
        np_ = self._dense(lengths, "lengths", torch.int32, (B,), keep)
        hp = self._dense(h0, "h0", f32, (B, H), keep)
        y = torch.empty(shape, dtype=dtype, device=dev)
        h_n = torch.empty((B, H), dtype=f32, device=dev)
        st = torch.empty((-(-T // RCU_LINREC_CHUNK), B, H), dtype=f32, device=dev) if states \
            else None
        _check(self.lib.rcu_linrec_forward(
            self.h, dt, 1 if batch_first else 0, T, B, H, xp, xl, rp, rl, ip, il, lp, c, np_, hp,
            y.data_ptr(), H, h_n.data_ptr(), st.data_ptr() if states else None,
            self._raw_stream()))
        return y, h_n, st

    def linrec_backward(self, dy, x, r, i, lam, states, c=8.0, lengths=None, dh_n=None,
                        batch_first=False, out=None, stream=None):
        """dx, dr, di (of dy's type), dlam [H] and dh0 [B, H].  x, r, i: the
        forward's inputs, or all three as act8_pack's (codes, exponents).  out:
        a contiguous tensor like dy but 3H wide, for the gradient of a fused
        projection: dx, dr, di are then its three parts."""
        if stream is not None:
            return self._on_stream(stream, self.linrec_backward, dy, x, r, i, lam, states, c,
                                   lengths, dh_n, batch_first, out)
        dtype, dt, shape = self._type(dy, "dy", 3)
        T, B, H = shape
        if batch_first:
            T, B = B, T
        keep, f32, dev = [], torch.float32, dy.device
        xp, xl, xe = self._saved(x, "x", dtype, shape, keep)
        rp, rl, re = self._saved(r, "r", dtype, shape, keep)
        ip, il, ie = self._saved(i, "i", dtype, shape, keep)
        if (xe is None) != (re is None) or (xe is None) != (ie is None):
            raise ValueError("x, r, i are all tensors or all 8-bit checkpoints")
        yp, yl = self._rows(dy, "dy", dtype, shape, keep)
        lp = self._dense(lam, "lam", f32, (H,), keep)
        np_ = self._dense(lengths, "lengths", torch.int32, (B,), keep)
        sp = self._dense(states, "states", f32, (-(-T // RCU_LINREC_CHUNK), B, H), keep)
        hp = self._dense(dh_n, "dh_n", f32, (B, H), keep)
        if out is None:
            dx = torch.empty(shape, dtype=dtype, device=dev)
            dr = torch.empty(shape, dtype=dtype, device=dev)
            di = torch.empty(shape, dtype=dtype, device=dev)
            ld = H
        else:
            if not isinstance(out, torch.Tensor) or not out.is_contiguous():
                raise ValueError("out must be a contiguous tensor")
            self._dense(out, "out", dtype, (*shape[:2], 3 * H), keep)
            dx, dr, di = out[..., :H], out[..., H:2 * H], out[..., 2 * H:]
            ld = 3 * H
        dlam = torch.empty((H,), dtype=f32, device=dev)
        dh0 = torch.empty((B, H), dtype=f32, device=dev)
        _check(self.lib.rcu_linrec_backward(
            self.h, dt, dt if xe is None else RCU_I8, 1 if batch_first else 0, T, B, H, xp, xl,
            rp, rl, ip, il, xe, re, ie, lp, c, np_, sp, yp, yl, hp, dx.data_ptr(),
            ld, dr.data_ptr(), ld, di.data_ptr(), ld, dlam.data_ptr(), dh0.data_ptr(),
            self._raw_stream()))
        return dx, dr, di, dlam, dh0

    def linrec_step(self, x, r, i, lam, state, c=8.0, slot=None, stream=None):
        """y [B, H] of one step of B requests; state [slots, H] is updated in
        place, at slot[b] (int32 [B], -1: takes no part; None: row b)."""
        if stream is not None:
            return self._on_stream(stream, self.linrec_step, x, r, i, lam, state, c, slot)
        dtype, dt, shape = self._type(x, "x", 2)
        B, H = shape
        keep, f32 = [], torch.float32
        if not isinstance(state, torch.Tensor) or state.dim() != 2 or not state.is_contiguous():
            raise ValueError("state must be a contiguous [slots, H] tensor")
        slots = state.shape[0]
        xp, xl = self._rows(x, "x", dtype, shape, keep)
        rp, rl = self._rows(r, "r", dtype, shape, keep)
        ip, il = self._rows(i, "i", dtype, shape, keep)
        lp = self._dense(lam, "lam", f32, (H,), keep)
        sp = self._dense(state, "state", f32, (slots, H), keep)
        tp = self._dense(slot, "slot", torch.int32, (B,), keep)
        y = torch.empty(shape, dtype=dtype, device=x.device)
        _check(self.lib.rcu_linrec_step(self.h, dt, B, H, xp, xl, rp, rl, ip, il, lp, c, sp, slots,
                                        tp, y.data_ptr(), H, self._raw_stream()))
        return y

    # ---- layer norm

    def layernorm_forward(self, x, weight=None, bias=None, eps=1e-5, residual=None, stream=None):
        """(y, mean, rstd) of x [..., n]; with a residual (y, sum, mean, rstd),
        sum = x + residual being what is normalised."""
        if stream is not None:
            return self._on_stream(stream, self.layernorm_forward, x, weight, bias, eps, residual)
        dtype, dt, shape = self._type(x, "x")
        n = shape[-1]
        rows = x.numel() // n if n else 0
        keep, f32, dev = [], torch.float32, x.device
        xp, xl = self._rows(x, "x", dtype, shape, keep)
        wp = self._dense(weight, "weight", f32, (n,), keep)
        bp = self._dense(bias, "bias", f32, (n,), keep)
        u, rp, rl, up = None, None, 0, None
        if residual is not None:
            rp, rl = self._rows(residual, "residual", dtype, shape, keep)
            u = torch.empty(shape, dtype=dtype, device=dev)
            up = u.data_ptr()
        y = torch.empty(shape, dtype=dtype, device=dev)
        lead = shape[:-1]
        mean = torch.empty(lead, dtype=f32, device=dev)
        rstd = torch.empty(lead, dtype=f32, device=dev)
        _check(self.lib.rcu_layernorm_forward(
            self.h, dt, rows, n, xp, xl, rp, rl, wp, bp, eps, y.data_ptr(), n, up, n,
            mean.data_ptr(), rstd.data_ptr(), self._raw_stream()))
        return (y, mean, rstd) if u is None else (y, u, mean, rstd)

    def layernorm_backward(self, dy, u, mean, rstd, weight=None, dsum=None, stream=None):
        """(du, dweight, dbias).  u: what the forward normalised (x, or its
        sum), or act8_pack's (codes, exponents) of it; dsum: the gradient that
        reaches u another way."""
        if stream is not None:
            return self._on_stream(stream, self.layernorm_backward, dy, u, mean, rstd, weight, dsum)
        dtype, dt, shape = self._type(dy, "dy")
        n = shape[-1]
        rows = dy.numel() // n if n else 0
        keep, f32, dev, lead = [], torch.float32, dy.device, shape[:-1]
        up, ul, ue = self._saved(u, "u", dtype, shape, keep)
        yp, yl = self._rows(dy, "dy", dtype, shape, keep)
        sp, sl = self._rows(dsum, "dsum", dtype, shape, keep) if dsum is not None else (None, 0)
        wp = self._dense(weight, "weight", f32, (n,), keep)
        mp = self._dense(mean, "mean", f32, lead, keep)
        rp = self._dense(rstd, "rstd", f32, lead, keep)
        du = torch.empty(shape, dtype=dtype, device=dev)
        dw = torch.empty((n,), dtype=f32, device=dev)
        db = torch.empty((n,), dtype=f32, device=dev)
        _check(self.lib.rcu_layernorm_backward(
            self.h, dt, dt if ue is None else RCU_I8, rows, n, yp, yl, up, ul, ue, wp, mp, rp, sp,
            sl, du.data_ptr(), n, dw.data_ptr(), db.data_ptr(), self._raw_stream()))
        return du, dw, db

    # ---- 8-bit activation checkpoints

    def act8_pack(self, x, stream=None):
        """(codes int8 [..., n], exponents int8 [..., ceil(n / 64)]) of x."""
        if stream is not None:
            return self._on_stream(stream, self.act8_pack, x)
        dtype, dt, shape = self._type(x, "x")
        n = shape[-1]
        rows = x.numel() // n if n else 0
        keep, dev = [], x.device
        xp, xl = self._rows(x, "x", dtype, shape, keep)
        codes = torch.empty(shape, dtype=torch.int8, device=dev)
        exps = torch.empty((*shape[:-1], -(-n // RCU_ACT8_BLOCK)), dtype=torch.int8, device=dev)
        _check(self.lib.rcu_act8_pack(self.h, dt, rows, n, xp, xl, codes.data_ptr(), n,
                                      exps.data_ptr(), self._raw_stream()))
        return codes, exps

    def act8_unpack(self, codes, exps, dtype=torch.float32, stream=None):
        """The values an 8-bit checkpoint stands for."""
        if stream is not None:
            return self._on_stream(stream, self.act8_unpack, codes, exps, dtype)
        dt = self._DTYPES.get(dtype)
        if dt is None:
            raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
        if not isinstance(codes, torch.Tensor) or codes.dim() < 1:
            raise ValueError("codes must be a tensor on a CUDA device")
        shape = codes.shape
        n = shape[-1]
        rows = codes.numel() // n if n else 0
        keep = []
        cp, cl, ep = self._saved((codes, exps), "x", None, shape, keep)
        y = torch.empty(shape, dtype=dtype, device=codes.device)
        _check(self.lib.rcu_act8_unpack(self.h, dt, rows, n, cp, cl, ep, y.data_ptr(), n,
                                        self._raw_stream()))
        return y

    # ---- handle

    def status(self, stream=None) -> int:
        """Synchronise and return the device status code (0 = ok); does not raise."""
        return self.lib.rcu_seq_get_status(self.h, _stream(stream))

    def set_attr(self, attr, value):
        _check(self.lib.rcu_seq_set_attr(self.h, attr, value))

    def launch_count(self) -> int:
        return self.lib.rcu_seq_last_launch_count(self.h)

    def profile(self) -> dict:
        """{call: (total_ms, calls)} recorded while RCU_ATTR_PROFILE is on."""
        out, i = {}, 0
        name, ms, n = ctypes.c_char_p(), ctypes.c_double(), ctypes.c_int64()
        while self.lib.rcu_seq_profile_entry(self.h, i, ctypes.byref(name), ctypes.byref(ms),
                                             ctypes.byref(n)) == RCU_OK:
            out[name.value.decode()] = (ms.value, n.value)
            i += 1
        return out

    def close(self):
        if self.h:
            self.lib.rcu_seq_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
