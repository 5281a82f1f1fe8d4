"""A small sequence mixer on this package's operators, as a model would run them.

One projection gives queries, keys, values, log-decays and angle increments.
``moments_rot_fwd`` sums the increments, ``moments_qk_fwd`` norms queries and keys for
each head and turns them into the frame of the cached states, ``moments_attn_fwd`` reads
the states out, and ``moments_fwd`` gives the states' moments, which a penalty in the
loss uses. Training runs all of it with gradients; serving runs the prompt in one
call and then single tokens on a pool of states.

    python examples/mixer.py        # a few training steps, then a prompt and its continuation
"""
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mamba_ssm_chunkwise_amd as M  # noqa: E402


class Rotation(torch.autograd.Function):
    """Cumulative angles [b,s,h,a] from per-token increments."""

    @staticmethod
    def forward(ctx, inc):
        ctx.save_for_backward(inc)
        return M.moments_rot_fwd(M.rot_desc(inc, M.ROT_PAIRWISE), inc)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_rot):
        (inc,) = ctx.saved_tensors
        return M.moments_rot_bwd(M.rot_desc(inc, M.ROT_PAIRWISE), inc, d_rot.contiguous())


class QueryKey(torch.autograd.Function):
    """Queries and keys, normed and turned; q and k may be columns of a projection."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, bq, bk, rot, heads):
        ctx.desc = M.qk_desc(q, k, heads, M.ROT_PAIRWISE, rot=rot)
        ctx.save_for_backward(q, k, wq, wk, bq, bk, rot)
        return M.moments_qk_fwd(ctx.desc, q, k, wq, wk, bq, bk, rot)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_qhat, d_khat):
        g = M.moments_qk_bwd(ctx.desc, *ctx.saved_tensors, d_qhat.contiguous(), d_khat.contiguous())
        return g["d_q"], g["d_k"], g["d_wq"], g["d_wk"], g["d_bq"], g["d_bk"], g["d_rot"], None


class Attention(torch.autograd.Function):
    """y and the last state of linear attention with a decay for each head."""

    @staticmethod
    def forward(ctx, x, khat, qhat, da, h0, lens):
        desc = M.attn_desc(x, khat, valid_lens=lens)
        y, last, saved = M.moments_attn_fwd_save(desc, x, khat, qhat, da, h0)
        ctx.desc = desc
        ctx.save_for_backward(x, khat, qhat, da, h0, lens, saved)   # lens too: the descriptor reads the buffer again
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y, d_last):
        x, khat, qhat, da, h0, _, saved = ctx.saved_tensors
        g = M.moments_attn_bwd_saved(ctx.desc, x, khat, qhat, da, h0, saved, d_y.contiguous(), d_last.contiguous())
        return g["d_xhat"], g["d_bhat"], g["d_qhat"], g["d_da"], g["d_h0"], None


class Moments(torch.autograd.Function):
    """Second moments of the de-rotated states, for a penalty on them."""

    @staticmethod
    def forward(ctx, x, khat, da, rot):
        ctx.desc = M.make_desc(x, khat, 1, x.shape[1], M.ROT_PAIRWISE, rope_dim=2 * rot.shape[3])
        ctx.save_for_backward(x, khat, da, rot)
        m2, m1 = M.moments_fwd(ctx.desc, x, khat, da, rot, None)
        ctx.m1_shape = m1.shape
        return m2

    @staticmethod
    @once_differentiable
    def backward(ctx, d_m2):
        x, khat, da, rot = ctx.saved_tensors
        g = M.moments_bwd(ctx.desc, x, khat, da, rot, None, d_m2.contiguous(), d_m2.new_zeros(ctx.m1_shape),
                          want=("xhat", "bhat", "da", "rot"))
        return g["d_xhat"], g["d_bhat"], g["d_da"], g["d_rot"]


class Mixer(torch.nn.Module):
    def __init__(self, width, heads=4, groups=2, p=32, r=64, angles=16, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.heads, self.groups, self.p, self.r, self.angles = heads, groups, p, r, angles
        self.cols = (groups * r, groups * r, heads * p, heads, heads * angles)   # q, k, x, decay, increments
        new = lambda *s, scale: torch.nn.Parameter(torch.randn(*s, device=device, dtype=dtype) * scale)  # noqa: E731
        self.w_in = new(width, sum(self.cols), scale=width ** -0.5)
        self.w_out = new(heads * p, width, scale=(heads * p) ** -0.5)
        par = lambda t: torch.nn.Parameter(t.to(device=device, dtype=torch.float32))  # noqa: E731
        self.wq, self.wk = par(torch.full((r,), r ** -0.5)), par(torch.full((r,), r ** -0.5))
        self.bq, self.bk = par(torch.zeros(heads, r)), par(torch.zeros(heads, r))

    def project(self, u):
        """Queries, keys (columns of the projection), values, log-decays, angle increments."""
        b, s, _ = u.shape
        q, k, x, dt, inc = (u @ self.w_in).split(self.cols, dim=-1)
        return (q.view(b, s, 1, self.groups, self.r), k.view(b, s, 1, self.groups, self.r),
                x.reshape(b, s, 1, self.heads, self.p).contiguous(), -torch.nn.functional.softplus(dt).contiguous(),
                (0.1 * inc).view(b, s, self.heads, self.angles).contiguous())

    def turned(self, q, k, rot):
        return QueryKey.apply(q, k, self.wq, self.wk, self.bq, self.bk, rot, self.heads)

    def out(self, y):
        return y.reshape(*y.shape[:2], -1) @ self.w_out

    def forward(self, u, penalty=False):
        q, k, x, da, inc = self.project(u)
        rot = Rotation.apply(inc)
        qhat, khat = self.turned(q, k, rot)
        y, _ = Attention.apply(x, khat, qhat, da, None, None)
        return self.out(y), (Moments.apply(x, khat, da, rot) if penalty else None)

    @torch.no_grad()
    def prompt(self, u, lens=None):
        """Outputs, and what a continuation needs: the states and the angles so far."""
        q, k, x, da, inc = self.project(u)
        rot = Rotation.apply(inc)
        qhat, khat = self.turned(q, k, rot)
        y, state = M.moments_attn_fwd(M.attn_desc(x, khat, valid_lens=lens), x, khat, qhat, da)
        at = torch.full((u.shape[0],), u.shape[1], device=u.device) if lens is None else lens.long()
        theta = rot.float()[torch.arange(u.shape[0], device=u.device), (at - 1).clamp(min=0)]
        return self.out(y), state, torch.where((at > 0)[:, None, None], theta, 0.0)

    @torch.no_grad()
    def token(self, u, state, theta, slots=None):
        """One token of each sequence u [b,1,width]; state and theta are updated in place: theta [b,heads,angles]
        row by row, state, a pool, at the rows' slots (without slots row by row too)."""
        q, k, x, da, inc = self.project(u)
        theta += inc[:, 0].float()
        rot = theta[:, None].to(u.dtype)
        qhat, khat = self.turned(q, k, rot)
        y = M.moments_attn_step(M.attn_desc(x, khat), x, khat, qhat, da, state, slots)
        return self.out(y)


def main():
    torch.manual_seed(0)
    mixer = Mixer(128)
    u = torch.randn(4, 512, 128, device="cuda", dtype=torch.bfloat16)
    target = torch.roll(u, 1, dims=1).float()
    opt = torch.optim.SGD(mixer.parameters(), lr=0.02)
    for step in range(5):
        out, m2 = mixer(u, penalty=True)
        loss = (out.float() - target).square().mean() + 1e-9 * m2.square().mean()
        opt.zero_grad()
        loss.backward()
        grads = M.grad_desc([p.grad for p in mixer.parameters()])
        M.moments_grad_clip(grads, M.moments_grad_norm(grads), 1.0)
        opt.step()
        print(f"step {step}: loss {loss.item():.5f}", flush=True)
    whole, _ = mixer(u[:, :200])
    _, state, theta = mixer.prompt(u[:, :190])
    tail = torch.cat([mixer.token(u[:, t:t + 1].contiguous(), state, theta) for t in range(190, 200)], 1)
    diff = (tail.float() - whole[:, 190:].float()).norm() / whole[:, 190:].float().norm()
    print(f"prompt of 190 and 10 single tokens against the whole sequence: {diff.item():.2e} apart", flush=True)


if __name__ == "__main__":
    main()
