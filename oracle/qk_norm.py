"""Norms of queries or keys for each head with the position rotation, and the
reverse-mode derivative, numpy fp64 (TEST INFRASTRUCTURE).

hat = M^T (n w + bias), n = x / sqrt(mean x^2 + eps), with M the de-rotation of the
moments path written out as an r x r matrix for each (token, head).
"""
import numpy as np

ROT_NONE, ROT_PAIRWISE, ROT_HALF, ROT_QUAT = 0, 1, 2, 3


def rotation_matrices(rot, kind, r):
    """M [..., r, r] of angles [..., a] or quaternions [..., J, 4], and dM / d rot
    [..., r, r] for each component (a list in the flattened order)."""
    lead = rot.shape[:-2] if kind == ROT_QUAT else rot.shape[:-1]
    M = np.broadcast_to(np.eye(r), lead + (r, r)).copy()
    D = []
    if kind == ROT_QUAT:
        basis = [np.eye(4),
                 np.array([[0, -1, 0, 0], [1, 0, 0, 0], [0, 0, 0, -1], [0, 0, 1, 0]], float),
                 np.array([[0, 0, -1, 0], [0, 0, 0, 1], [1, 0, 0, 0], [0, -1, 0, 0]], float),
                 np.array([[0, 0, 0, -1], [0, 0, -1, 0], [0, 1, 0, 0], [1, 0, 0, 0]], float)]
        for j in range(rot.shape[-2]):
            sl = slice(4 * j, 4 * j + 4)
            M[..., sl, sl] = sum(rot[..., j, e, None, None] * basis[e] for e in range(4))
            for e in range(4):
                d = np.zeros((r, r))
                d[sl, sl] = basis[e]
                D.append(np.broadcast_to(d, lead + (r, r)))
        return M, D
    for i in range(rot.shape[-1]):
        a, b = (2 * i, 2 * i + 1) if kind == ROT_PAIRWISE else (i, r // 2 + i)
        c, s = np.cos(rot[..., i]), np.sin(rot[..., i])
        M[..., a, a], M[..., a, b], M[..., b, a], M[..., b, b] = c, s, -s, c
        d = np.zeros(lead + (r, r))
        d[..., a, a], d[..., a, b], d[..., b, a], d[..., b, b] = -s, c, -c, -s
        D.append(d)
    return M, D


def _parts(x, w, bias, rot, kind, h, eps):
    b, s, c, g, r = x.shape
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * rstd
    u = np.repeat(n * w, h // g, axis=3)
    if bias is not None:
        u = u + bias
    if kind == ROT_NONE:
        return rstd, n, u, None, None
    M, D = rotation_matrices(rot, kind, r)
    return rstd, n, u, np.broadcast_to(M, (b, s, h, r, r)), D


def qk_fwd(x, w, bias, rot, kind, h, eps):
    _, _, u, M, _ = _parts(x, w, bias, rot, kind, h, eps)
    return u if M is None else np.einsum("bshji,bschj->bschi", M, u)


def qk_bwd(x, w, bias, rot, kind, h, eps, d):
    """d_x, d_w, d_bias, d_rot (None without a rotation) of one tensor."""
    b, s, c, g, r = x.shape
    rstd, n, u, M, D = _parts(x, w, bias, rot, kind, h, eps)
    du, d_rot = d, None
    if M is not None:
        du = np.einsum("bshji,bschi->bschj", M, d)
        d_rot = np.stack([np.einsum("bshji,bschj,bschi->bsh", np.broadcast_to(m, (b, s, h, r, r)), u, d)
                          for m in D], -1)
        if rot.shape[2] == 1 and h != 1:
            d_rot = d_rot.sum(2, keepdims=True)
        d_rot = d_rot.reshape(rot.shape)
    d_bias = du.sum((0, 1, 2))
    dg = du.reshape(b, s, c, g, h // g, r).sum(4)
    d_w = (dg * n).sum((0, 1, 2, 3))
    dn = dg * w
    d_x = rstd * (dn - n * (dn * n).mean(-1, keepdims=True))
    return d_x, d_w, d_bias, d_rot
