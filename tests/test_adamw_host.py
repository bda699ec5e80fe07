"""What the optimizer object refuses (no GPU needed)."""
import types

import pytest
import torch

from recurrent_cell_unroll_gb300.adamw import AdamW


def test_a_parameter_given_twice_is_refused():
    p, q = torch.zeros(3), torch.zeros(3)
    opt = AdamW([p, q], ops=object())
    assert [len(t) for t in (opt.params, opt.m, opt.v)] == [2, 2, 2]
    with pytest.raises(ValueError, match="twice"):
        AdamW([p, q, p], ops=object())
    with pytest.raises(ValueError, match="twice"):
        AdamW(iter([q, q]), ops=object())


def test_a_step_is_not_captured(monkeypatch):
    """Its number is the host's: a replay would repeat it."""
    calls = []
    ops = types.SimpleNamespace(adamw_step=lambda *a, **k: calls.append(a[4]))
    opt = AdamW([torch.zeros(3)], ops=ops)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    opt.step()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="captured"):
        opt.step()
    assert calls == [1] and opt.steps == 1


def test_a_step_on_another_stream(monkeypatch):
    on = []

    def on_stream(stream, call, *args):
        on.append(stream)
        return call(*args)
    calls = []
    ops = types.SimpleNamespace(adamw_step=lambda *a, **k: calls.append(k["lr"]), _on_stream=on_stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: on == [])
    opt = AdamW([torch.zeros(3)], ops=ops)
    opt.step(lr=0.5, stream=7)
    assert on == [7] and calls == [0.5] and opt.steps == 1
