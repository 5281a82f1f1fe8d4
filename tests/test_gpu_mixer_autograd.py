"""What examples/mixer.py leaves to autograd: tensors held for the backward, and where
gradients end."""
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from test_gpu_mixer import _example

pytestmark = pytest.mark.gpu


def _inputs(s=5, h=2, g=1, p=16, r=24):
    f = lambda *shape: torch.randn(*shape, device="cuda").requires_grad_()  # noqa: E731
    return f(1, s, 1, h, p), f(1, s, 1, g, r), f(1, s, 1, g, r), -torch.rand(1, s, h, device="cuda"), f(1, h, p, r)


def test_a_state_changed_before_the_backward_is_noticed():
    """The initial state, a cached one, is updated in place by single tokens between forward and backward."""
    x, k, q, da, h0 = _inputs()
    y, last = _example().Attention.apply(x, k, q, da, h0, None)
    one = [v[:, :1].detach().contiguous() for v in (x, k, q, da)]
    M.moments_attn_step(M.attn_desc(one[0], one[1]), *one, h0.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("name", ["Attention", "QueryKey", "Rotation", "Moments"])
def test_second_order_gradients_are_refused(name):
    """The gradients have no graph of their own: asking for theirs is an error, not a silent zero."""
    ex = _example()
    x, k, q, da, h0 = _inputs()
    w, bias = torch.ones(24, device="cuda"), torch.zeros(2, 24, device="cuda")
    rot = torch.randn(1, 5, 2, 6, device="cuda").requires_grad_()
    khat = torch.randn(1, 5, 1, 2, 24, device="cuda")
    out = {"Attention": lambda: ex.Attention.apply(x, k, q, da, h0, None)[0],
           "QueryKey": lambda: ex.QueryKey.apply(k, q, w, w, bias, bias, rot, 2)[0],
           "Rotation": lambda: ex.Rotation.apply(rot),
           "Moments": lambda: ex.Moments.apply(x, khat, da, rot)}[name]()
    leaf = rot if name == "Rotation" else (k if name == "QueryKey" else x)
    (g,) = torch.autograd.grad(out.square().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (g.square().sum() + leaf.sum()).backward()
