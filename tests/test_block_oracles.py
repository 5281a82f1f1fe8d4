"""The oracles of the gated recurrence and of layer norm, pinned without a GPU: automatic
differentiation of the definitions in 64 bits, differences, and closed forms."""
import numpy as np
import pytest
import torch

from oracle import gated_rec, layer_norm

RNG = np.random.default_rng(11)


def _case(kind, b=2, s=9, w=5, z=True):
    x, g, zz, dy = (RNG.standard_normal((b, s, w)) for _ in range(4))
    g = -np.abs(g) if kind == gated_rec.LOG else 2 * g
    return x, g, zz if z else None, RNG.standard_normal((b, w)), dy, RNG.standard_normal((b, w))


def _torch_rec(x, g, z, h0, kind):
    h, ys = h0, []
    for t in range(x.shape[1]):
        a = torch.exp(g[:, t]) if kind == gated_rec.LOG else torch.sigmoid(g[:, t])
        u = x[:, t]
        if kind == gated_rec.MIX:
            u = (1 - a) * u
        elif kind == gated_rec.UNIT:
            u = torch.sqrt(1 - a * a) * u
        h = a * h + u
        ys.append(h if z is None else h * torch.nn.functional.silu(z[:, t]))
    return torch.stack(ys, 1), h


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("z", [True, False])
def test_recurrence_against_autograd(kind, z):
    x, g, zz, h0, dy, dl = _case(kind, z=z)
    o = gated_rec.rec(x, g, zz, h0, kind, d_y=dy, d_h_last=dl)
    t = {n: torch.tensor(v, requires_grad=True) for n, v in (("x", x), ("g", g), ("z", zz), ("h0", h0)) if v is not None}
    y, last = _torch_rec(t["x"], t["g"], t.get("z"), t["h0"], kind)
    ((y * torch.tensor(dy)).sum() + (last * torch.tensor(dl)).sum()).backward()
    np.testing.assert_allclose(o["y"], y.detach(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(o["h_last"], last.detach(), rtol=1e-12, atol=1e-12)
    for n in t:
        np.testing.assert_allclose(o["d_" + n], t[n].grad, rtol=1e-10, atol=1e-11)


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_recurrence_padding_clearing_and_pieces(kind):
    x, g, z, h0, dy, dl = _case(kind, b=3)
    whole = gated_rec.rec(x, g, z, h0, kind)
    first = gated_rec.rec(x[:, :4], g[:, :4], z[:, :4], h0, kind)
    rest = gated_rec.rec(x[:, 4:], g[:, 4:], z[:, 4:], first["h_last"], kind)
    np.testing.assert_allclose(np.concatenate([first["y"], rest["y"]], 1), whole["y"], rtol=1e-13)
    o = gated_rec.rec(x, g, z, h0, kind, lens=[5, 0, 9], d_y=dy, d_h_last=dl)
    assert not o["y"][0, 5:].any() and not o["d_g"][1].any()
    np.testing.assert_array_equal(o["h_last"][1], h0[1])
    np.testing.assert_array_equal(o["d_h0"][1], dl[1])
    g[:, 4] = -np.inf                     # a new sequence from there on, whatever stood before
    x[:, 2] = np.inf
    fresh = gated_rec.rec(x[:, 4:], g[:, 4:], z[:, 4:], None, kind)
    np.testing.assert_array_equal(gated_rec.rec(x, g, z, h0, kind)["y"][:, 4:], fresh["y"])


def test_recurrence_constant_gate():
    """A mean of the state and x settles at x; a gate of unit variance keeps that of white noise."""
    x, g = np.full((1, 400, 1), 3.0), np.full((1, 400, 1), 2.0)
    assert abs(gated_rec.rec(x, g, None, None, gated_rec.MIX)["h_last"][0, 0] - 3.0) < 1e-12
    noise = RNG.standard_normal((1, 400, 4000))
    var = gated_rec.rec(noise, np.broadcast_to(g, noise.shape), None, None, gated_rec.UNIT)["h_last"].var()
    assert abs(var - 1.0) < 0.1           # of 4000 draws: sd sqrt(2 / 4000) = 0.022


@pytest.mark.parametrize("res,bias", [(True, True), (False, False)])
def test_layer_norm_against_autograd(res, bias):
    n, w = 7, 12
    t = {"x": torch.randn(n, w, dtype=torch.float64), "weight": torch.randn(w, dtype=torch.float64)}
    if res:
        t["res"] = torch.randn(n, w, dtype=torch.float64)
    if bias:
        t["bias"] = torch.randn(w, dtype=torch.float64)
    t = {k: v.requires_grad_() for k, v in t.items()}
    dy, ds = torch.randn(n, w, dtype=torch.float64), torch.randn(n, w, dtype=torch.float64)
    s = t["x"] + t["res"] if res else t["x"]
    y = torch.nn.functional.layer_norm(s, (w,), t["weight"], t.get("bias"), 1e-3)
    ((y * dy).sum() + ((s * ds).sum() if res else 0.0)).backward()
    a = {k: v.detach().numpy() for k, v in t.items()}
    o = layer_norm.ln(a["x"], a.get("res"), a["weight"], a.get("bias"), 1e-3, dy.numpy(), ds.numpy() if res else None)
    np.testing.assert_allclose(o["y"], y.detach(), rtol=1e-11, atol=1e-12)
    for k in ("x", "res"):
        if k in t:
            np.testing.assert_allclose(o["d_s"], t[k].grad, rtol=1e-10, atol=1e-12)
    for k in ("weight", "bias"):
        if k in t:
            np.testing.assert_allclose(o["d_" + k], t[k].grad, rtol=1e-10, atol=1e-12)
