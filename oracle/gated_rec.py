"""The gated linear recurrence over channels and its reverse-mode derivative, token by
token, numpy fp64 (TEST INFRASTRUCTURE).

h[t] = a[t] h[t-1] + u[t], y[t] = h[t] z[t] sigma(z[t]) (or h[t]), with a decay and an
input from the gate. A decay of zero forgets whatever stood before, values that are not
finite among it. Padded tokens (t >= lens[b]) are skipped.

With ``bounds`` every result comes with what float32 arithmetic may be off by, in the same
walk. One rounding is U = 2^-24 of its result; the exponential, reciprocal and root
instructions are good to one unit in the last place, 2 U. M is the sum of magnitudes that
a state is made of; each token may add the roundings of its decay, of the product that
hands the state on (through runs, waves and segments: 4) and of its input. 2^-125 is for what
underflows on the way; a state of zero that meets an input of zero stays exactly that.
"""
import numpy as np

LOG, MIX, UNIT = 0, 1, 2
U = 2.0 ** -24


def _sigma(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def gate(g, kind):
    """a, b = 1 - a, f and the relative errors of each in units of U."""
    m = np.minimum(np.abs(g), 88.0)
    if kind == LOG:
        one = np.ones_like(g)
        with np.errstate(over="ignore"):
            return np.exp(g), 0.0 * one, one, 2 + 2 * m, 0.0 * one, 0.0 * one
    a, b = _sigma(g), _sigma(-g)
    e = np.exp(-m)                                # the smaller side is e r, r = 1 / (1 + e), the larger 1 - e r
    re = 2 + 2 * m if kind == MIX else 5 + 2 * m  # UNIT: a square of exp(-m / 2), 2 (2 + m) + 1
    rr = e / (1 + e) * re + 3
    small = re + rr + 1
    large = e * small + 1
    ra, rb = np.where(g < 0, small, large), np.where(g < 0, large, small)
    if kind == MIX:
        return a, b, b, ra, rb, rb
    f = np.sqrt(b * (1 + a))
    # sqrt(r (1 + a)), times exp(-m / 2) where g is not negative
    return a, b, f, ra, rb, 0.5 * (rr + a / (1 + a) * ra + 2) + 2 + np.where(g < 0, 0, 2 + m + 1)


def _silu(z):
    """sigma(z), z sigma(z) and their relative error in units of U."""
    s = _sigma(z)
    r = (1 - s) * (2 + 2 * np.minimum(np.abs(z), 88.0)) + 3
    return s, z * s, r + 1


def _times(a, h):
    with np.errstate(invalid="ignore"):
        return np.where(a == 0, 0.0, a * h)


def rec(x, g, z, h0, kind, lens=None, d_y=None, d_h_last=None, bounds=False):
    """dict of y, h_last and, with d_y, d_x, d_g, d_z, d_h0, each fp64; with ``bounds`` also
    of the errors that float32 arithmetic may leave, under the same names with "e_" before."""
    b, s, w = x.shape
    lens = [s] * b if lens is None else [int(min(max(v, 0), s)) for v in lens]
    names = ["y"] + (["d_x", "d_g"] + (["d_z"] if z is not None else []) if d_y is not None else [])
    o = {p + n: np.zeros((b, s, w)) for n in names for p in ("", "e_")}
    o.update({p + n: np.zeros((b, w)) for n in ("h_last", "d_h0") for p in ("", "e_")})
    for i, n in enumerate(lens):
        xi, gi = x[i, :n], g[i, :n]
        a, bb, f, ra, rb, rf = gate(gi, kind)
        if kind == LOG:
            u, ru = xi, 0.0 * xi
        else:
            u, ru = f * xi, rf + 1
        H, M, E = np.zeros((n + 1, w)), np.zeros((n + 1, w)), np.zeros((n + 1, w))
        if h0 is not None:
            H[0], M[0] = h0[i], np.abs(h0[i])
        for t in range(n):
            H[t + 1] = _times(a[t], H[t]) + u[t]
            if bounds:
                M[t + 1] = a[t] * M[t] + np.abs(u[t])
                E[t + 1] = a[t] * E[t] + U * ((ra[t] + 4) * a[t] * M[t] + (ru[t] + 4) * np.abs(u[t]))
                E[t + 1] += np.where((M[t] > 0) | (u[t] != 0), 2.0 ** -125, 0.0)
        o["h_last"][i], o["e_h_last"][i] = H[n], E[n]
        if z is None:
            o["y"][i, :n], o["e_y"][i, :n] = H[1:], E[1:]
        else:
            sg, sl, rs = _silu(z[i, :n])
            o["y"][i, :n] = H[1:] * sl
            o["e_y"][i, :n] = E[1:] * np.abs(sl) + U * (rs + 1) * np.abs(H[1:] * sl)
        if d_y is None:
            continue
        dy = d_y[i, :n]
        src, rsrc = (dy, 0.0 * dy) if z is None else (dy * sl, rs + 1)
        c = np.zeros(w) if d_h_last is None else d_h_last[i].astype(float)
        mc, ec = np.abs(c), np.zeros(w)
        for t in range(n - 1, -1, -1):
            d = src[t] + c
            ed = ec + U * rsrc[t] * np.abs(src[t]) + U * (np.abs(src[t]) + mc)
            hp, ep, at = H[t], E[t], a[t]
            if kind == LOG:
                o["d_x"][i, t], o["e_d_x"][i, t] = d, ed
                q, eq = hp, ep
            else:
                o["d_x"][i, t], o["e_d_x"][i, t] = f[t] * d, f[t] * ed + U * (rf[t] + 1) * np.abs(f[t] * d)
                if kind == MIX:
                    q = bb[t] * (hp - xi[t])
                    eq = bb[t] * (ep + U * (np.abs(hp) + np.abs(xi[t]))) + U * (rb[t] + 1) * np.abs(q)
                else:
                    k = f[t] / (1 + at)
                    rk = rf[t] + at / (1 + at) * ra[t] + 4
                    q = bb[t] * hp - at * xi[t] * k
                    eq = bb[t] * ep + U * (rb[t] + 2) * np.abs(bb[t] * hp) + U * (ra[t] + rk + 3) * np.abs(at * xi[t] * k)
            o["d_g"][i, t] = _times(at, q * d)
            o["e_d_g"][i, t] = at * (np.abs(q) * ed + np.abs(d) * eq + ed * eq) + U * (ra[t] + 2) * np.abs(at * q * d)
            # a decay below 2^-126 is taken as zero: a q d is then off by itself, |a q d| < 2^-126 |q d|
            o["e_d_g"][i, t] += 2.0 ** -126 * np.abs(q * d)
            if z is not None:
                zt, st = z[i, t], sg[t]
                sp = st * (1 + zt * (1 - st))
                esp = U * (rs[t] * np.abs(sp) + st * np.abs(zt) * (rs[t] * st + 2) + 4 * st * (1 + np.abs(zt) * (1 - st)))
                o["d_z"][i, t] = dy[t] * H[t + 1] * sp
                o["e_d_z"][i, t] = np.abs(dy[t]) * (E[t + 1] * np.abs(sp) + np.abs(H[t + 1]) * esp) + 3 * U * np.abs(
                    dy[t] * H[t + 1] * sp)
            ec = at * (ec + U * rsrc[t] * np.abs(src[t])) + U * (ra[t] + 4) * at * (np.abs(src[t]) + mc)
            ec += np.where((mc > 0) | (src[t] != 0), 2.0 ** -125, 0.0)
            c, mc = _times(at, d), at * (np.abs(src[t]) + mc)
        o["d_h0"][i], o["e_d_h0"][i] = c, ec
    return o
