"""A stack of gated recurrent blocks on this package's operators, as a model would run them.

Each block norms the float32 residual stream after adding what the block before gave it
(``moments_ln_fwd``), projects the normed rows to inputs, gates and output gates, runs the
recurrence over them (``moments_rec_fwd_save``, columns of the projection as they are) and
projects back. Training clips the gradients by their global norm (``moments_grad_norm``,
``moments_grad_clip``); serving runs the prompt in one call and then single tokens on pools
of states (``moments_rec_step``).

    python examples/recurrent.py        # a few training steps, then a prompt and its continuation
"""
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mamba_ssm_chunkwise_amd as M  # noqa: E402


class AddNorm(torch.autograd.Function):
    """y and the new residual stream of layer norm over x + res."""

    @staticmethod
    def forward(ctx, x, res, weight, bias):
        ctx.desc = M.ln_desc(x, residual=True)
        y, total = M.moments_ln_fwd(ctx.desc, x, weight, bias, res)
        ctx.save_for_backward(total, weight, bias)
        return y, total

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y, d_sum):
        total, weight, bias = ctx.saved_tensors
        g = M.moments_ln_bwd(ctx.desc, total, weight, bias, d_y.contiguous(), d_sum.contiguous())
        return g["d_x"], g["d_res"], g["d_weight"], g["d_bias"]


class Recurrence(torch.autograd.Function):
    """y and the last state of the gated recurrence; x, g and z may be columns of a projection."""

    @staticmethod
    def forward(ctx, x, g, z, h0, gate, lens):
        ctx.desc = M.rec_desc(x, g, z, gate, valid_lens=lens)
        y, last, saved = M.moments_rec_fwd_save(ctx.desc, x, g, z, h0)
        ctx.save_for_backward(x, g, z, h0, lens, saved)   # lens too: the descriptor reads the buffer again
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y, d_last):
        x, g, z, h0, _, saved = ctx.saved_tensors
        d = M.moments_rec_bwd_saved(ctx.desc, x, g, z, h0, saved, d_y.contiguous(), d_last.contiguous())
        return d["d_x"], d["d_g"], d["d_z"], d["d_h0"], None, None


class Stack(torch.nn.Module):
    def __init__(self, width, blocks=2, inner=64, gate=M.GATE_UNIT, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.width, self.blocks, self.inner, self.gate = width, blocks, inner, gate
        new = lambda *s, scale: torch.nn.Parameter(torch.randn(*s, device=device, dtype=dtype) * scale)  # noqa: E731
        par = lambda t: torch.nn.Parameter(t.to(device=device, dtype=torch.float32))  # noqa: E731
        each = lambda f: torch.nn.ParameterList([f() for _ in range(blocks)])  # noqa: E731
        self.w_in = each(lambda: new(width, 3 * inner, scale=width ** -0.5))
        self.w_out = each(lambda: new(inner, width, scale=inner ** -0.5))
        self.weight, self.bias = each(lambda: par(torch.ones(width))), each(lambda: par(torch.zeros(width)))
        # gates whose channels forget over one token up to some hundreds
        self.shift = par(torch.linspace(0.0, 5.0, inner))

    def project(self, i, y):
        x, g, z = (y @ self.w_in[i]).split(self.inner, dim=-1)
        return x, (g + self.shift).to(y.dtype), z

    def forward(self, u, lens=None):
        """What the last block adds to the stream, and the stream, for u [b,s,width]."""
        x, res = u, torch.zeros(u.shape, dtype=torch.float32, device=u.device)
        for i in range(self.blocks):
            y, res = AddNorm.apply(x, res, self.weight[i], self.bias[i])
            y, _ = Recurrence.apply(*self.project(i, y), None, self.gate, lens)
            x = y @ self.w_out[i]
        return x, res

    @torch.no_grad()
    def prompt(self, u, lens=None):
        """Outputs as forward's, and the states [blocks][b,inner] that a continuation needs."""
        x, res, states = u, torch.zeros(u.shape, dtype=torch.float32, device=u.device), []
        for i in range(self.blocks):
            y, res = M.moments_ln_fwd(M.ln_desc(x, residual=True), x, self.weight[i], self.bias[i], res, sum=res)
            x, g, z = self.project(i, y)
            y, last = M.moments_rec_fwd(M.rec_desc(x, g, z, self.gate, valid_lens=lens), x, g, z)
            states.append(last)
            x = y @ self.w_out[i]
        return x, res, states

    @torch.no_grad()
    def token(self, u, states, slots=None):
        """One token of each sequence u [b,1,width] on the pools of states, updated in place."""
        x, res = u, torch.zeros(u.shape, dtype=torch.float32, device=u.device)
        for i in range(self.blocks):
            y, res = M.moments_ln_fwd(M.ln_desc(x, residual=True), x, self.weight[i], self.bias[i], res, sum=res)
            x, g, z = self.project(i, y)
            y = M.moments_rec_step(M.rec_desc(x, g, z, self.gate), x, g, z, states[i], slots)
            x = y @ self.w_out[i]
        return x, res


def main():
    torch.manual_seed(0)
    stack = Stack(128)
    u = torch.randn(4, 512, 128, device="cuda", dtype=torch.bfloat16)
    target = torch.roll(u, 1, dims=1).float()
    opt = torch.optim.SGD(stack.parameters(), lr=0.5)
    for step in range(5):
        x, res = stack(u)
        loss = (x.float() + res - target).square().mean()
        opt.zero_grad()
        loss.backward()
        grads = M.grad_desc([p.grad for p in stack.parameters()])
        norm = M.moments_grad_norm(grads)
        M.moments_grad_clip(grads, norm, 1.0)
        opt.step()
        print(f"step {step}: loss {loss.item():.5f}, gradients' norm {norm.item():.4f}", flush=True)
    whole, _ = stack(u[:, :200].contiguous())
    _, _, states = stack.prompt(u[:, :190].contiguous())
    tail = torch.cat([stack.token(u[:, t:t + 1].contiguous(), states)[0] for t in range(190, 200)], 1)
    diff = (tail.float() - whole[:, 190:].float()).norm() / whole[:, 190:].float().norm()
    print(f"prompt of 190 and 10 single tokens against the whole sequence: {diff.item():.2e} apart", flush=True)


if __name__ == "__main__":
    main()
