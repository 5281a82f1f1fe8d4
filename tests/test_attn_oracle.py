"""The 64-bit oracles of linear attention and of the norms with rotation, pinned
on the CPU: their gradients against central differences, the recurrence against
its closed double sum, a sequence against the same cut in two, groups of heads
against repeated keys, and the queries' frame against the de-rotated states."""
import numpy as np
import pytest

from oracle import attn_seq, qk_norm

RNG = np.random.default_rng(5)


def _case(b=2, s=5, c=2, h=4, g=2, p=3, r=6):
    f = RNG.standard_normal
    return {"x": f((b, s, c, h, p)), "k": f((b, s, c, g, r)), "q": f((b, s, c, g, r)), "da": -np.abs(f((b, s, h))),
            "h0": f((b, h, p, r))}


def _diff(f, a, eps=1e-6):
    """Central differences of the scalar f with respect to the array a (in place)."""
    out = np.zeros(a.shape)
    for i in np.ndindex(a.shape):
        v = a[i]
        a[i] = v + eps
        hi = f()
        a[i] = v - eps
        lo = f()
        a[i] = v
        out[i] = (hi - lo) / (2 * eps)
    return out


@pytest.mark.parametrize("lens", [None, [3, 0]])
def test_attention_gradients_against_differences(lens):
    t = _case(s=4)
    d_y, d_last = RNG.standard_normal(t["x"].shape), RNG.standard_normal(t["h0"].shape)
    lens = None if lens is None else np.array(lens)
    live = np.ones(t["x"].shape[:2], bool) if lens is None else np.arange(4)[None] < lens[:, None]

    def loss():
        y, last = attn_seq.attn_fwd(t["x"], t["k"], t["q"], t["da"], t["h0"], lens)
        return (y * d_y * live[:, :, None, None, None]).sum() + (last * d_last).sum()

    got = attn_seq.attn_bwd(t["x"], t["k"], t["q"], t["da"], t["h0"], d_y, d_last, lens)
    for name, key in (("x", "d_xhat"), ("k", "d_bhat"), ("q", "d_qhat"), ("da", "d_da"), ("h0", "d_h0")):
        # differences at 1e-6 carry about 1e-9 of rounding; values are of order 1 to 100
        np.testing.assert_allclose(got[key], _diff(loss, t[name]), rtol=1e-6, atol=1e-6, err_msg=name)


def test_attention_is_its_double_sum():
    t = _case(g=4)
    y, _ = attn_seq.attn_fwd(t["x"], t["k"], t["q"], t["da"], None)
    a = t["da"].cumsum(1)
    for tt in range(5):
        ref = np.zeros(y[:, tt].shape)
        for j in range(tt + 1):
            w = np.exp(a[:, tt] - a[:, j])
            dot = np.einsum("bchr,bdhr->bcdh", t["q"][:, tt], t["k"][:, j])
            ref += np.einsum("bh,bcdh,bdhp->bchp", w, dot, t["x"][:, j])
        np.testing.assert_allclose(y[:, tt], ref, rtol=1e-12, atol=1e-12)


def test_attention_in_two_pieces_and_by_groups():
    t = _case(s=7)
    whole, last = attn_seq.attn_fwd(t["x"], t["k"], t["q"], t["da"], t["h0"])
    one, mid = attn_seq.attn_fwd(*(t[n][:, :3] for n in ("x", "k", "q", "da")), t["h0"])
    two, end = attn_seq.attn_fwd(*(t[n][:, 3:] for n in ("x", "k", "q", "da")), mid)
    np.testing.assert_allclose(np.concatenate([one, two], 1), whole, rtol=1e-13)
    np.testing.assert_allclose(end, last, rtol=1e-13)
    rep = attn_seq.attn_fwd(t["x"], np.repeat(t["k"], 2, 3), np.repeat(t["q"], 2, 3), t["da"], t["h0"])[0]
    np.testing.assert_array_equal(rep, whole)


ROTS = [(qk_norm.ROT_NONE, 0), (qk_norm.ROT_PAIRWISE, 3), (qk_norm.ROT_HALF, 2), (qk_norm.ROT_QUAT, 1)]


def _rot(kind, width, lead):
    if kind == qk_norm.ROT_NONE:
        return None
    return RNG.standard_normal(lead + ((width, 4) if kind == qk_norm.ROT_QUAT else (width,)))


@pytest.mark.parametrize("kind,width", ROTS)
@pytest.mark.parametrize("rot_h", [1, 4])
def test_norm_gradients_against_differences(kind, width, rot_h):
    b, s, c, g, h, r = 1, 2, 2, 2, 4, 6
    x, w, bias = RNG.standard_normal((b, s, c, g, r)), RNG.standard_normal(r), RNG.standard_normal((h, r))
    rot, d = _rot(kind, width, (b, s, rot_h)), RNG.standard_normal((b, s, c, h, r))

    def loss():
        return (qk_norm.qk_fwd(x, w, bias, rot, kind, h, 1e-3) * d).sum()

    got = qk_norm.qk_bwd(x, w, bias, rot, kind, h, 1e-3, d)
    for a, v in zip((x, w, bias, rot), got):
        if a is not None:
            np.testing.assert_allclose(v, _diff(loss, a), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("kind,width", ROTS[1:])
def test_queries_read_the_derotated_state(kind, width):
    """<h, M^T q> = <M h, q>: the frame the moments path de-rotates its states to."""
    q, rot, hst = RNG.standard_normal((1, 1, 1, 1, 6)), _rot(kind, width, (1, 1, 1)), RNG.standard_normal(6)
    hat = qk_norm.qk_fwd(q, np.ones(6), None, rot, kind, 1, 0.0)[0, 0, 0, 0]
    n = q[0, 0, 0, 0] / np.sqrt((q ** 2).mean())
    M = qk_norm.rotation_matrices(rot, kind, 6)[0][0, 0, 0]
    assert abs(hst @ hat - (M @ hst) @ n) < 1e-13
