"""Layer norm of rows with a residual and its reverse-mode derivative, numpy fp64 (TEST
INFRASTRUCTURE), with what float32 arithmetic may be off by.

One rounding is U = 2^-24 of its result. A sum of w values goes through at most K = 64
additions in a row (16 in a thread, 6 across a wave, 15 across waves, and the products), so
it is off by K U times the sum of magnitudes.
"""
import numpy as np

U = 2.0 ** -24
K = 64


def ln(x, res, weight, bias, eps, d_y=None, d_sum=None, row_adds=64):
    """dict of y, sum and, with d_y, d_s (of x and of res alike), d_weight, d_bias, each with its
    bound under "e_". ``row_adds``: additions in a row of the sums over rows."""
    o = {}
    s = x if res is None else x + res
    es = 0.0 * s if res is None else U * np.abs(s)
    o["sum"], o["e_sum"] = s, es
    d = s - s.mean(-1, keepdims=True)
    mean = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
    # the first mean's error (taken about the row's first value), which the second takes out
    slip = K * U * (mean(np.abs(s)) + np.abs(s[:, :1]))
    ed = es + mean(es) + U * (2 * np.abs(d) + slip) + (K + 3) * U * mean(np.abs(d) + slip)
    var = mean(d * d)
    rstd = 1.0 / np.sqrt(var + eps)
    evar = mean(2 * np.abs(d) * ed + ed * ed) + K * U * mean((np.abs(d) + ed) ** 2)
    rr = 0.5 * evar / (var + eps) + 4 * U           # relative, of rstd
    xhat = d * rstd
    ex = ed * rstd + np.abs(xhat) * rr + U * np.abs(xhat)
    b = 0.0 if bias is None else bias
    o["y"] = xhat * weight + b
    o["e_y"] = np.abs(weight) * ex + 2 * U * (np.abs(xhat * weight) + np.abs(b))
    if d_y is None:
        return o
    gy = d_y * weight
    m1, m2 = mean(gy), mean(gy * xhat)
    em1 = (K + 2) * U * mean(np.abs(gy))
    em2 = mean(np.abs(gy) * ex) + (K + 4) * U * mean(np.abs(gy) * (np.abs(xhat) + ex)) + rr * np.abs(m2)
    inner = gy - m1 - xhat * m2
    o["d_s"] = rstd * inner
    o["e_d_s"] = rstd * (U * np.abs(gy) + em1 + np.abs(xhat) * em2 + ex * (np.abs(m2) + em2)
                         + 4 * U * (np.abs(gy) + np.abs(m1) + np.abs(xhat * m2))) + (rr + 2 * U) * np.abs(o["d_s"])
    if d_sum is not None:
        o["d_s"] = o["d_s"] + d_sum
        o["e_d_s"] = o["e_d_s"] + U * np.abs(o["d_s"])
    o["d_weight"], o["d_bias"] = (d_y * xhat).sum(0), d_y.sum(0)
    o["e_d_weight"] = (np.abs(d_y) * ex).sum(0) + (row_adds + 3) * U * (np.abs(d_y) * (np.abs(xhat) + ex)).sum(0)
    o["e_d_bias"] = (row_adds + 3) * U * np.abs(d_y).sum(0)
    return o
