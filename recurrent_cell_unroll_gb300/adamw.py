"""AdamW over a list of parameters in one call a step (SeqOps.adamw_step), with its
states in fp32 or, of larger tensors, in 8 bits.
"""
from __future__ import annotations

import torch

from . import binding


class AdamW:
    """Decoupled weight decay Adam of float32 or bfloat16 leaves on one device.

    state_bits 8: tensors of `min_8bit` values or more hold both moments in 8 bits
    (a quarter of the memory; small ones, norms and biases, stay in fp32).  A step
    takes the leaves' .grad, leaves out those that have none, and counts once for
    all.  `ops`: the SeqOps to call (made when None); one stream at a time uses it.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits=32, min_8bit=4096, seed=0, ops=None):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        self.params = list(params)
        if len({id(p) for p in self.params}) < len(self.params):
            raise ValueError("a parameter is given twice: a step would update it in two places at once")
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.seed, self.steps = seed, 0
        self.ops = binding.SeqOps() if ops is None else ops
        self.m, self.v = [], []
        for p in self.params:
            for held, signed in ((self.m, True), (self.v, False)):
                zero = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                held.append(self.ops.state8_pack(zero, signed)
                            if state_bits == 8 and p.numel() >= min_8bit else zero)

    @torch.no_grad()
    def step(self, lr=None, scale=None, stream=None):
        """One step; lr in the place of the optimizer's; scale: a float32 on the
        device that gradients are multiplied by (clipping, loss scaling).  Not to be
        captured into a graph: its number is counted here, so each replay would be the
        same step (SeqOps.adamw_step can read it from the device)."""
        if stream is not None:
            return self.ops._on_stream(stream, self.step, lr, scale)
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("AdamW.step counts its steps on the host and cannot be captured; call "
                               "SeqOps.adamw_step with step (and lr) as tensors on the device")
        self.ops.adamw_step(self.params, [p.grad for p in self.params], self.m, self.v, self.steps + 1,
                            lr=self.lr if lr is None else lr, betas=self.betas, eps=self.eps,
                            weight_decay=self.weight_decay, scale=scale, seed=self.seed)
        self.steps += 1

    def zero_grad(self):
        for p in self.params:
            p.grad = None

    def state_dict(self) -> dict:
        """Steps and states as they are held, of tensors that further steps update in
        place."""
        return {"steps": self.steps, "m": list(self.m), "v": list(self.v)}

    def load_state_dict(self, state: dict):
        """Copies a state_dict of an optimizer that holds its states alike."""
        def parts(held):
            return [t for s in held for t in (s if isinstance(s, tuple) else (s,))]
        pairs = []
        for mine, other in ((self.m, state["m"]), (self.v, state["v"])):
            a, b = parts(mine), parts(other)
            if len(a) != len(b) or any(x.shape != y.shape or x.dtype != y.dtype for x, y in zip(a, b)):
                raise ValueError("the states are held in another way, or of other parameters")
            pairs += zip(a, b)
        for x, y in pairs:
            x.copy_(y)
        self.steps = int(state["steps"])
