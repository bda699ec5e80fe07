"""The selective-scan stack: layer norm, short convolution, scan and AdamW together, as a
model trains and serves with them."""
import pytest
import torch

import ssm_ref as ref
from recurrent_cell_unroll_gb300 import adamw, ssm_block

pytestmark = pytest.mark.gpu


def plain(net, blocks, x, lengths):
    """The stack's forward by the formulas, in 64 bits."""
    u, v, after = x, torch.zeros_like(x), ([], [])
    zero = torch.zeros(x.shape[1], net.taps - 1, net.hidden, dtype=torch.float64)
    for b in blocks:
        u = u + v
        d = u - u.mean(-1, keepdim=True)
        n = d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5) * b["weight"] + b["bias"]
        xs, z = (n @ b["w_in"]).chunk(2, -1)
        xs, window = ref.conv(xs, b["conv"], b["conv_bias"], True, lengths, zero)
        r, bw, cw = (xs @ b["w_x"]).split([net.rank, net.states, net.states], -1)
        y, h, _ = ref.scan(xs, r @ b["w_dt"], b["a_log"], bw, cw, b["d"], b["dt_bias"], z, lengths, None)
        v = y @ b["w_out"]
        after[0].append(window)
        after[1].append(h)
    return u + v, torch.stack(after[0]), torch.stack(after[1])


def test_stack_gradients():
    """Against torch autograd on the same formulas in 64 bits.  Products in fp32 (TF32 is
    off by default) round some 2^-20 of their terms' scale, and pass through two blocks."""
    net = ssm_block.SSMStack(2, 24, 40, states=6, dtype=torch.float32)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(70, 3, 24, generator=g)
    lengths = torch.tensor([70, 33, 1])
    y, (window, h) = net.forward(x.cuda(), lengths=lengths.int().cuda())
    out = (y, window, h)
    ws = [torch.randn(t.shape, generator=g) for t in out]
    sum((t * w.cuda()).sum() for t, w in zip(out, ws)).backward()
    leaves = [{k: t.detach().cpu().double().requires_grad_() for k, t in b.items()} for b in net.blocks]
    want = plain(net, leaves, x.double(), lengths)
    sum((t * w.double()).sum() for t, w in zip(want, ws)).backward()
    for got, w in zip(out, want):
        assert float((got.detach().cpu().double() - w.detach()).abs().max()) <= 1e-4 * float(w.detach().abs().max())
    for b, r in zip(net.blocks, leaves):
        for k, t in b.items():
            off = float((t.grad.cpu().double() - r[k].grad).abs().max())
            assert off <= 1e-4 * float(r[k].grad.abs().max()), (k, off)


@pytest.mark.parametrize("opt8", [False, True])
def test_trains_and_serves(opt8):
    losses, off = ssm_block.main(["--steps", "20"] + (["--opt8"] if opt8 else []))
    assert all(v == v for v in losses)
    assert off <= 2e-2  # two passes of bf16 activations


def test_serving_with_slots():
    """Requests at slots of a table, some of them waiting: as rows of their own."""
    net = ssm_block.SSMStack(2, 32, 48, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(12, 3, 32, generator=g, device="cuda")
    with torch.no_grad():
        whole, _ = net.forward(x)
        table = net.zero_state(7)
        slot = torch.tensor([6, 2, 4], dtype=torch.int32, device="cuda")
        for t in range(12):
            y = net.step(x[t], table, slot)
            assert float((y - whole[t]).abs().max()) <= 1e-4 * float(whole.abs().max())
        assert not any(bool(t[:, [0, 1, 3, 5]].any()) for t in table)


def test_a_prompt_in_pieces():
    net = ssm_block.SSMStack(1, 32, 48, dtype=torch.float32)
    x = torch.randn(90, 2, 32, device="cuda")
    with torch.no_grad():
        whole, after = net.forward(x)
        state, parts = None, []
        for piece in x.split([1, 2, 40, 47]):
            y, state = net.forward(piece, state)
            parts.append(y)
    assert float((torch.cat(parts) - whole).abs().max()) <= 1e-4 * float(whole.abs().max())
    for a, b in zip(state, after):
        assert float((a - b).abs().max()) <= 1e-4 * float(b.abs().max())


def test_training_step_as_a_graph():
    """Forward, backward and the optimizer's step, captured and replayed, move the
    parameters as eager steps do."""
    def fresh():
        net = ssm_block.SSMStack(1, 32, 48, dtype=torch.float32)
        m, v = ([torch.zeros_like(p) for p in net.parameters()] for _ in range(2))
        return net, m, v
    x = torch.randn(40, 2, 32, device="cuda")
    step = torch.ones(1, dtype=torch.int32, device="cuda")

    def train(net, m, v, count):
        y, _ = net.forward(x)
        grads = torch.autograd.grad(y.square().mean(), net.parameters())
        net.ops.adamw_step([p.detach() for p in net.parameters()], grads, m, v, count, lr=1e-3)
    eager = fresh()
    for t in (1, 2, 3):
        train(*eager, t)
    graphed = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train(*graphed, step)  # the first step, eager
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train(*graphed, step)
    for t in (2, 3):
        step.fill_(t)
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager[0].parameters(), graphed[0].parameters()):
        assert torch.equal(a, b)


def test_optimizer_object():
    g = torch.Generator().manual_seed(4)
    start = [torch.randn(s, generator=g) for s in ((70, 70), (33,), (64, 2))]

    def leaves():
        return [t.cuda().requires_grad_() for t in start]
    a, b = leaves(), leaves()
    mine, other = adamw.AdamW(a, lr=1e-2), torch.optim.AdamW(b, lr=1e-2, fused=False, foreach=False)
    for k in range(5):
        for p, q in zip(a, b):
            q.grad = torch.randn(q.shape, generator=g).cuda()
            p.grad = q.grad.clone()
        mine.step()
        other.step()
    for p, q in zip(a, b):  # five updates of lr, each good to 1e-6 of it
        assert float((p - q).abs().max()) <= 5 * 1e-2 * 1e-6 + 2.0 ** -22 * float(q.abs().max())
    eight = adamw.AdamW(a, lr=1e-2, state_bits=8)
    assert isinstance(eight.m[0], tuple) and isinstance(eight.m[1], torch.Tensor)
    eight.step()
    again = adamw.AdamW(a, lr=1e-2, state_bits=8)
    again.load_state_dict(eight.state_dict())
    assert again.steps == 1 and torch.equal(again.v[0][0], eight.v[0][0])
    with pytest.raises(ValueError):
        again.load_state_dict(mine.state_dict())
    with pytest.raises(ValueError):
        adamw.AdamW(a, state_bits=16)


def test_a_graph_that_saved_a_parameter_refuses_to_go_on():
    p = torch.randn(8, 8, device="cuda", requires_grad=True)
    opt = adamw.AdamW([p])
    x = torch.randn(8, 8, device="cuda", requires_grad=True)
    loss = (x @ p).sum()
    p.grad = torch.ones_like(p)
    opt.step()
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
