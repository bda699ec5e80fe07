"""Graphs that have saved what the AdamW step changes in place, and graphs of the step itself."""
import pytest
import torch

from recurrent_cell_unroll_gb300 import adamw, binding

pytestmark = pytest.mark.gpu


def test_a_graph_that_saved_a_copy_refuses_to_go_on():
    ops = binding.SeqOps()
    p = torch.randn(8, 8, device="cuda")
    copy = p.bfloat16()
    x = torch.randn(8, 8, device="cuda").bfloat16().requires_grad_()
    loss = (x @ copy).sum()
    zeros = [torch.zeros_like(p) for _ in range(2)]
    ops.adamw_step([p], [torch.ones_like(p)], zeros[:1], zeros[1:], 1, copies=[copy])
    assert torch.equal(copy, p.bfloat16()) and ops.status() == 0
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    ops.close()


def test_the_optimizer_object_is_not_captured():
    p = torch.randn(64, device="cuda", requires_grad=True)
    p.grad = torch.ones_like(p)
    opt = adamw.AdamW([p])
    opt.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    opt.step(stream=side)
    torch.cuda.synchronize()
    before = p.detach().clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = before * 2
        with pytest.raises(RuntimeError, match="captured"):
            opt.step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, before * 2) and torch.equal(p.detach(), before) and opt.steps == 2
