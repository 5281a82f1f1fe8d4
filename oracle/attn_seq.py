"""Linear attention with a decay for each head, token by token, and its adjoint,
numpy fp64 (TEST INFRASTRUCTURE).

Per (b, head): h[t] = e^{da[t]} h[t-1] + sum_c x[t,c] (outer) k[t,c], y[t,c] = h[t] q[t,c],
head hi using key group hi / (h/g). Tokens past a sequence's length do nothing and
have zero outputs and gradients. The adjoint carries G[t], the cotangent of h[t], and
takes d_da[t] = e^{da[t]} <G[t], h[t-1]> straight from its definition (the states are
all kept: small sizes only).
"""
import numpy as np


def _setup(x, k, q, da, h0, lens):
    b, s, c, h, p = x.shape
    g, r = k.shape[3:]
    grp = np.arange(h) // (h // g)
    H = np.zeros((b, h, p, r)) if h0 is None else h0.astype(np.float64).copy()
    lens = np.full(b, s) if lens is None else np.clip(lens, 0, s)
    return b, s, c, h, p, g, r, grp, H, lens


def attn_fwd(x, k, q, da, h0=None, lens=None, keep=False):
    b, s, c, h, p, g, r, grp, H, lens = _setup(x, k, q, da, h0, lens)
    y = np.zeros((b, s, c, h, p))
    states = np.zeros((b, s + 1, h, p, r)) if keep else None
    for bi in range(b):
        S = H[bi]
        if keep:
            states[bi, 0] = S
        for t in range(lens[bi]):
            S = np.exp(da[bi, t])[:, None, None] * S + np.einsum("chp,chr->hpr", x[bi, t], k[bi, t][:, grp])
            y[bi, t] = np.einsum("hpr,chr->chp", S, q[bi, t][:, grp])
            if keep:
                states[bi, t + 1] = S
        H[bi] = S
    return (y, H, states) if keep else (y, H)


def attn_bwd(x, k, q, da, h0, d_y, d_last=None, lens=None):
    b, s, c, h, p, g, r, grp, _, n = _setup(x, k, q, da, h0, lens)
    _, _, st = attn_fwd(x, k, q, da, h0, lens, keep=True)
    out = {"d_xhat": np.zeros(x.shape), "d_bhat": np.zeros(k.shape), "d_qhat": np.zeros(q.shape),
           "d_da": np.zeros(da.shape), "d_h0": np.zeros((b, h, p, r))}
    for bi in range(b):
        G = np.zeros((h, p, r)) if d_last is None else d_last[bi].astype(np.float64).copy()
        for t in range(n[bi] - 1, -1, -1):
            kt, qt = k[bi, t][:, grp], q[bi, t][:, grp]
            G = G + np.einsum("chp,chr->hpr", d_y[bi, t], qt)
            dq = np.einsum("chp,hpr->chr", d_y[bi, t], st[bi, t + 1])
            dk = np.einsum("chp,hpr->chr", x[bi, t], G)
            out["d_xhat"][bi, t] = np.einsum("hpr,chr->chp", G, kt)
            out["d_qhat"][bi, t] = dq.reshape(c, g, h // g, r).sum(2)
            out["d_bhat"][bi, t] = dk.reshape(c, g, h // g, r).sum(2)
            G = np.exp(da[bi, t])[:, None, None] * G
            out["d_da"][bi, t] = (G * st[bi, t]).sum((1, 2))
        out["d_h0"][bi] = G
    return out
