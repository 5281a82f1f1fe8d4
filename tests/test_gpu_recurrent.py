"""Layer norm, the gated recurrence and the gradients' clipping together, as
examples/recurrent.py runs them: its gradients against automatic differentiation of the same
stack written out in 64 bits on the host, their norm and clipped values, and a prompt with its
continuation by single tokens against the whole sequence.

float32 throughout: 1e-4 leaves room for the library's matrix products and for the chain of two
blocks, each operator within a few 1e-6."""
import importlib.util
import os

import pytest
import torch

import mamba_ssm_chunkwise_amd as M

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example(name="recurrent"):
    spec = importlib.util.spec_from_file_location(name + "_example", os.path.join(ROOT, "examples", name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _plain(p, u, blocks, inner, gate):
    """x and the stream in 64 bits on the host, token by token."""
    x, res = u, torch.zeros_like(u)
    for i in range(blocks):
        res = x + res
        d = res - res.mean(-1, keepdim=True)
        y = d / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt() * p[f"weight.{i}"] + p[f"bias.{i}"]
        xs, g, z = (y @ p[f"w_in.{i}"]).split(inner, dim=-1)
        a = torch.exp(g + p["shift"]) if gate == M.GATE_LOG else torch.sigmoid(g + p["shift"])
        f = {M.GATE_LOG: torch.ones_like(a), M.GATE_MIX: 1 - a, M.GATE_UNIT: (1 - a * a).sqrt()}[gate]
        h, hs = torch.zeros_like(xs[:, 0]), []
        for t in range(u.shape[1]):
            h = a[:, t] * h + f[:, t] * xs[:, t]
            hs.append(h)
        x = (torch.stack(hs, 1) * torch.nn.functional.silu(z)) @ p[f"w_out.{i}"]
    return x, res


@pytest.mark.parametrize("gate", [M.GATE_MIX, M.GATE_UNIT])
def test_training_step_against_64_bits(gate):
    torch.manual_seed(5)
    stack = _example().Stack(24, blocks=2, inner=20, gate=gate, dtype=torch.float32)
    u = torch.randn(2, 150, 24, device="cuda")
    d_x, d_res = torch.randn(2, 150, 24, device="cuda"), torch.randn(2, 150, 24, device="cuda")
    x, res = stack(u)
    ((x * d_x).sum() + (res * d_res).sum()).backward()
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in stack.named_parameters()}
    rx, rr = _plain(p, u.double().cpu(), 2, 20, gate)
    ((rx * d_x.double().cpu()).sum() + (rr * d_res.double().cpu()).sum()).backward()
    pairs = {"x": (x, rx), "res": (res, rr)}
    pairs.update({k: (v.grad, p[k].grad) for k, v in stack.named_parameters()})
    for name, (got, ref) in pairs.items():
        e = ((got.detach().double().cpu() - ref.detach()).norm() / ref.detach().norm()).item()
        print(f"[compare] {name}: {e:.2e}", flush=True)
        assert e <= 1e-4, (name, e)
    want = torch.stack([v.grad.square().sum() for v in p.values()]).sum().sqrt().item()
    grads = M.grad_desc([v.grad for v in stack.parameters()])
    norm = M.moments_grad_norm(grads)
    assert abs(norm.item() - want) <= 1e-4 * want
    M.moments_grad_clip(grads, norm, 0.5)
    for k, v in stack.named_parameters():
        ref = p[k].grad * min(1.0, 0.5 / (want + 1e-6))
        assert (v.grad.double().cpu() - ref).norm() <= 2e-4 * ref.norm(), k


def test_prompt_and_single_tokens():
    torch.manual_seed(6)
    stack = _example().Stack(24, blocks=2, inner=20, dtype=torch.float32)
    u = torch.randn(3, 60, 24, device="cuda")
    whole, stream = stack(u)
    lens = torch.tensor([50, 0, 33], dtype=torch.int32, device="cuda")
    out, _, states = stack.prompt(u[:, :50].contiguous(), lens)
    for b, n in enumerate(lens.tolist()):
        assert torch.allclose(out[b, :n], whole[b, :n], atol=1e-4, rtol=1e-4)
    rows, pos = torch.arange(3, device="cuda"), lens.long()
    pools = [torch.zeros(5, 20, device="cuda") for _ in states]      # the sequences' states at slots of a pool
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    for pool, s in zip(pools, states):
        pool[slots.long()] = s
    for _ in range(10):                       # each sequence goes on from its own length
        y, res = stack.token(u[rows, pos][:, None].contiguous(), pools, slots)
        assert torch.allclose(y[:, 0], whole[rows, pos], atol=1e-4, rtol=1e-4)
        assert torch.allclose(res[:, 0], stream[rows, pos], atol=1e-4, rtol=1e-4)
        pos = pos + 1


def test_the_example_runs():
    _example().main()
    _example("mixer").main()


def test_second_order_gradients_are_refused():
    """The gradients have no graph of their own: asking for theirs is an error, not a silent zero."""
    ex = _example()
    f = lambda *shape: torch.randn(*shape, device="cuda").requires_grad_()  # noqa: E731
    x, g, z = f(1, 6, 8), f(1, 6, 8), f(1, 6, 8)
    weight, bias = f(8), f(8)
    for leaf, out in ((x, ex.Recurrence.apply(x, g, z, None, M.GATE_MIX, None)[0]),
                      (weight, ex.AddNorm.apply(x, z, weight, bias)[0])):
        (d,) = torch.autograd.grad(out.square().sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (d.square().sum() + leaf.sum()).backward()


def test_a_state_changed_before_the_backward_is_noticed():
    """The initial state, a cached one, is updated in place by single tokens between forward and backward."""
    ex = _example()
    f = lambda *shape: torch.randn(*shape, device="cuda").requires_grad_()  # noqa: E731
    x, g, z, h0 = f(1, 6, 8), f(1, 6, 8), f(1, 6, 8), f(1, 8)
    y, _ = ex.Recurrence.apply(x, g, z, h0, M.GATE_MIX, None)
    one = [v[:, :1].detach().contiguous() for v in (x, g, z)]
    M.moments_rec_step(M.rec_desc(*one, M.GATE_MIX), *one, h0.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_training_step_captured():
    """Forward and backward of the stack in a graph, replayed on new inputs, against the eager step."""
    torch.manual_seed(8)
    stack = _example().Stack(32, blocks=2, inner=24, dtype=torch.float32)
    u = torch.randn(2, 140, 32, device="cuda")
    params = list(stack.parameters())

    def step():
        x, res = stack(u)
        return torch.autograd.grad(x.square().sum() + res.square().sum(), params)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2, 3):
        torch.manual_seed(seed)
        u.copy_(torch.randn(2, 140, 32, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.allclose(a, b, rtol=1e-5, atol=1e-5 * b.abs().max().item())
