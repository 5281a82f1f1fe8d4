"""Comparison with an oracle's result and its bound, element by element."""
import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # a rounding of the output, relative


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(name, got, ref, err):
    """|got - ref| within err plus the rounding of the output's type (2^-133 for its smallest values)."""
    half = HALF[got.dtype]
    g = np64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{name}: non-finite values"
    if g.size == 0:
        return
    lim = err + (np.abs(ref) + err) * half + 2.0 ** -133
    off = np.abs(g - ref) / lim
    at = np.unravel_index(np.argmax(off), off.shape)
    print(f"[compare] {name}: at most {off[at]:.3f} of its bound, at {at}: {g[at]:.9g} for {ref[at]:.9g}", flush=True)
    assert off[at] <= 1.0, f"{name} at {at}: {g[at]!r} for {ref[at]!r}, bound {lim[at]:.3e}"


def same(a, b):
    """The same bits, NaN among them."""
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
