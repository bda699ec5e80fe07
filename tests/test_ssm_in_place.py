"""What the AdamW step and the single steps change in place, autograd is told of: a graph
that has saved such a tensor refuses to go on (no GPU needed)."""
import types

import pytest
import torch

from recurrent_cell_unroll_gb300 import binding


def saved_by(weight):
    """The loss of a graph that has saved `weight`."""
    return (torch.ones(2, 4, requires_grad=True) @ weight).sum()


def test_parameters_and_their_copies():
    p, c = (torch.randn(4, 3) for _ in range(2))
    losses = [saved_by(p), saved_by(c)]
    binding._tensors().changed([p], [torch.ones(4, 3)], [c])
    for loss in losses:
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()


def test_tensors_that_a_step_leaves_out_have_not_changed():
    p, c, q = (torch.randn(4, 3) for _ in range(3))
    losses = [saved_by(p), saved_by(c), saved_by(q)]
    binding._tensors().changed([p, q], [None, torch.ones(4, 3)], [c, None])
    losses[0].backward()
    losses[1].backward()
    with pytest.raises(RuntimeError, match="inplace"):
        losses[2].backward()
    binding._tensors().changed([p], [torch.ones(4, 3)], None)
    with torch.inference_mode():
        t = torch.zeros(3)
    binding._tensors().changed([t], [t], [t])


def test_lists_only():
    for args in ((1, [], None), ([], 1, None), ([], [], 1)):
        with pytest.raises(TypeError):
            binding._tensors().changed(*args)


def steps():
    """Each single step on host tensors, its kernel left out: name, call, table."""
    ops = object.__new__(binding.SeqOps)
    ops.h, ops.device, ops._raw_stream = None, -1, lambda: None
    ops.lib = types.SimpleNamespace(**{f"rcu_{n}_step": lambda *a: 0 for n in ("conv", "selscan", "linrec")})
    x, w, b, al = torch.zeros(2, 4), torch.zeros(4, 3), torch.zeros(2, 5), torch.zeros(4, 5)
    window, states, held = torch.zeros(6, 2, 4), torch.zeros(6, 4, 5), torch.zeros(6, 4)
    return [("conv", lambda: ops.conv_step(x, w, window), window),
            ("selscan", lambda: ops.selscan_step(x, x, al, b, b, states), states),
            ("linrec", lambda: ops.linrec_step(x, x, x, torch.zeros(4), held), held)]


@pytest.mark.parametrize("k", range(3), ids=["conv", "selscan", "linrec"])
def test_tables_of_single_steps(k):
    _, call, table = steps()[k]
    leaf = torch.ones(table.shape, requires_grad=True)
    loss = (leaf * table).sum()   # saves the table
    part = (leaf[:, :1] * table[:, :1]).sum()   # saves a view of it
    with torch.no_grad():
        call()
    for graph in (loss, part):
        with pytest.raises(RuntimeError, match="inplace"):
            graph.backward()
    with torch.inference_mode():
        _, call, table = steps()[k]
        call()
