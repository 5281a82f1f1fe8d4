"""The operators together, as examples/mixer.py runs them: its gradients against
automatic differentiation of the same mixer written out in 64 bits on the host, and a
prompt with its continuation by single tokens against the whole sequence.

float32 throughout: 1e-4 leaves room for the library's matrix products and for the chain
of five operators, each within 1e-5."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("mixer_example", os.path.join(ROOT, "examples", "mixer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _plain(p, u, heads, groups, cols, n, r, a):
    """out and m2 in 64 bits on the host, token by token."""
    b, s, _ = u.shape
    q, k, x, dt, inc = (u @ p["w_in"]).split(cols, dim=-1)
    x, da = x.reshape(b, s, heads, n), -torch.nn.functional.softplus(dt)
    rot = (0.1 * inc).reshape(b, s, heads, a).cumsum(1)

    def norm(t, w, bias):
        t = t.reshape(b, s, groups, r)
        t = t / (t.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w
        return t.repeat_interleave(heads // groups, 2) + bias

    def turn(t, sign):
        e, o = t[..., 0:2 * a:2], t[..., 1:2 * a:2]
        c, sn = rot.cos(), sign * rot.sin()
        return torch.cat([torch.stack([e * c - o * sn, e * sn + o * c], -1).flatten(-2), t[..., 2 * a:]], -1)

    qn, khat = norm(q, p["wq"], p["bq"]), turn(norm(k, p["wk"], p["bk"]), 1.0)
    H, ys, m2 = torch.zeros(b, heads, n, r, dtype=u.dtype), [], 0.0
    for t in range(s):
        H = da[:, t].exp()[..., None, None] * H + x[:, t, :, :, None] * khat[:, t, :, None, :]
        e, o = H[..., 0:2 * a:2], H[..., 1:2 * a:2]           # the de-rotated state, read by the plain query
        c, sn = rot[:, t, :, None].cos(), rot[:, t, :, None].sin()
        C = torch.cat([torch.stack([e * c + o * sn, o * c - e * sn], -1).flatten(-2), H[..., 2 * a:]], -1)
        ys.append((C * qn[:, t, :, None]).sum(-1))
        m2 = m2 + C.transpose(-1, -2) @ C
    return torch.stack(ys, 1).reshape(b, s, -1) @ p["w_out"], m2


def test_training_step_against_64_bits():
    torch.manual_seed(3)
    mixer = _example().Mixer(24, heads=4, groups=2, p=16, r=24, angles=6, dtype=torch.float32)
    u = torch.randn(2, 70, 24, device="cuda")
    d_out, d_m2 = torch.randn(2, 70, 24, device="cuda"), torch.randn(2, 4, 24, 24, device="cuda")
    out, m2 = mixer(u, penalty=True)
    ((out * d_out).sum() + (m2 * d_m2).sum()).backward()
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in mixer.named_parameters()}
    ro, rm = _plain(p, u.double().cpu(), 4, 2, mixer.cols, 16, 24, 6)
    ((ro * d_out.double().cpu()).sum() + (rm * d_m2.double().cpu()).sum()).backward()
    pairs = {"out": (out, ro), "m2": (m2, rm)}
    pairs.update({k: (v.grad, p[k].grad) for k, v in mixer.named_parameters()})
    for name, (got, ref) in pairs.items():
        e = ((got.detach().double().cpu() - ref.detach()).norm() / ref.detach().norm()).item()
        print(f"[compare] {name}: {e:.2e}", flush=True)
        assert e <= 1e-4, (name, e)


def test_prompt_and_single_tokens():
    torch.manual_seed(4)
    mixer = _example().Mixer(24, heads=4, groups=2, p=16, r=24, angles=6, dtype=torch.float32)
    u = torch.randn(3, 60, 24, device="cuda")
    whole, _ = mixer(u)
    lens = torch.tensor([50, 0, 33], dtype=torch.int32, device="cuda")
    out, state, theta = mixer.prompt(u[:, :50].contiguous(), lens)
    for b, n in enumerate(lens.tolist()):
        assert torch.allclose(out[b, :n], whole[b, :n], atol=1e-4, rtol=1e-4)
    pos = lens.long()
    for _ in range(10):                       # each sequence goes on from its own length
        tok = u[torch.arange(3, device="cuda"), pos][:, None].contiguous()
        y = mixer.token(tok, state, theta)
        assert torch.allclose(y[:, 0], whole[torch.arange(3, device="cuda"), pos], atol=1e-4, rtol=1e-4)
        pos = pos + 1
