"""What the optimizer object refuses (no GPU needed)."""
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
