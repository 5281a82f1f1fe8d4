"""GPU parity of the norms of queries and keys with the rotation, and of their
gradients, with the 64-bit oracle (oracle/qk_norm.py).

Tolerances. float32: a handful of roundings of 2^-24 for each value and sums of at
most 128 terms, those over tokens in double: 1e-5. bfloat16: one rounding of the
result, at most 2^-9 of it (2^-8 of the largest magnitude leaves room for the fp32
part); float32 gradients of parameters are held to the float32 bound.
"""
import numpy as np
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from oracle import qk_norm
from parity_util import max_err, rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-5, BF16: 2.0 ** -8}
EPS = 1e-5


def _np(x):
    return None if x is None else x.detach().double().cpu().numpy()


def _check(name, got, ref, tol):
    got = _np(got)
    assert np.all(np.isfinite(got)), f"{name}: non-finite values"
    e, m = rel_err(got, ref), max_err(got, ref)
    print(f"[compare] {name}: normwise {e:.2e} max-elementwise {m:.2e}", flush=True)
    assert e <= tol and m <= tol, f"{name}: {e:.2e}/{m:.2e} above {tol:.1e}"


def _make(b, s, c, h, g, r, kind, width, dtype, rot_h=None, bias=True, stride=(0, 0), seed=1, scale=1.0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    f = lambda *shape: torch.randn(*shape, device=DEV, generator=gen)  # noqa: E731
    t = {}
    row = c * g * r
    for n, st in zip(("q", "k"), stride):
        t[n] = f(b, s, st or row).to(dtype)[:, :, :row].view(b, s, c, g, r)
        t["w" + n] = 1.0 + 0.2 * f(r)
        t["b" + n] = 0.3 * f(h, r) if bias else None
        t["d_%shat" % n] = f(b, s, c, h, r).to(dtype)
    rot_h = h if rot_h is None else rot_h
    t["rot"] = None
    if kind == M.ROT_QUAT:
        t["rot"] = f(b, s, rot_h, width, 4).to(dtype)          # any quaternions, not only unit ones
    elif kind != M.ROT_NONE:
        t["rot"] = (f(b, s, rot_h, width) * scale).to(dtype)
    return t


def _all(t, h, kind):
    d = M.qk_desc(t["q"], t["k"], h, kind, rot=t["rot"], eps=EPS)
    args = [t[n] for n in ("q", "k", "wq", "wk", "bq", "bk", "rot")]
    hats = M.moments_qk_fwd(d, *args)
    got = M.moments_qk_bwd(d, *args, t["d_qhat"], t["d_khat"])
    o = {k: _np(v) for k, v in t.items()}
    rot = 0.0
    for i, n in enumerate(("q", "k")):
        a = (o[n], o["w" + n], o["b" + n], o["rot"], kind, h, EPS)
        _check(n + "hat", hats[i], qk_norm.qk_fwd(*a), TOL[t["q"].dtype])
        d_x, d_w, d_b, d_r = qk_norm.qk_bwd(*a, o["d_%shat" % n])
        _check("d_" + n, got["d_" + n], d_x, TOL[t["q"].dtype])
        _check("d_w" + n, got["d_w" + n], d_w, TOL[F32])
        if t["b" + n] is None:
            assert got["d_b" + n] is None
        else:
            _check("d_b" + n, got["d_b" + n], d_b, TOL[F32])
        rot = rot + d_r if d_r is not None else None
    if rot is None:
        assert got["d_rot"] is None
    else:
        _check("d_rot", got["d_rot"], rot, TOL[t["q"].dtype])
    return hats, got


KINDS = [(M.ROT_NONE, 0), (M.ROT_PAIRWISE, 5), (M.ROT_HALF, 6), (M.ROT_QUAT, 3)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind,width", KINDS)
@pytest.mark.parametrize("c,h,g", [(1, 1, 1), (2, 4, 4), (3, 6, 2), (4, 8, 1), (1, 7, 1), (2, 24, 2)])
def test_heads_and_channels(dtype, kind, width, c, h, g):
    print(f"[case] kind={kind} c={c} h={h} g={g} {dtype}", flush=True)
    _all(_make(2, 9, c, h, g, 24, kind, width, dtype, seed=c + h), h, kind)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [k for k, _ in KINDS])
@pytest.mark.parametrize("r", [4, 7, 16, 30, 45, 64, 66, 90, 96, 128])
def test_row_widths(dtype, kind, r):
    """Odd and unaligned rows; the whole width turned, and one pair or block."""
    if kind == M.ROT_HALF and r % 2:
        pytest.skip("half-split rows are even")
    full = 0 if kind == M.ROT_NONE else r // 4 if kind == M.ROT_QUAT else r // 2
    for width in sorted({full, min(1, full)}):
        print(f"[case] kind={kind} r={r} width={width} {dtype}", flush=True)
        _all(_make(1, 6, 2, 4, 2, r, kind, width, dtype, seed=r), 4, kind)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind,width", KINDS[1:])
@pytest.mark.parametrize("h,g,r", [(4, 4, 32), (6, 2, 128), (16, 1, 64)])
def test_one_rotation_for_all_heads(dtype, kind, width, h, g, r):
    _all(_make(2, 11, 2, h, g, r, kind, width, dtype, rot_h=1, seed=h), h, kind)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("stride", [(100, 0), (104, 64), (65, 66), (72, 200)])
def test_columns_of_a_projection(dtype, stride):
    """Token strides wider than the rows, aligned and not."""
    _all(_make(2, 7, 1, 4, 2, 32, M.ROT_PAIRWISE, 8, dtype, stride=stride, seed=4), 4, M.ROT_PAIRWISE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("h,r", [(32, 128), (100, 128), (128, 64), (96, 20)])
def test_one_group_of_many_heads(dtype, h, r):
    """More heads on one key than a wave has row slots."""
    print(f"[case] h={h} r={r} {dtype}", flush=True)
    _all(_make(1, 5, 1, h, 1, r, M.ROT_PAIRWISE, 3, dtype, seed=h), h, M.ROT_PAIRWISE)


@pytest.mark.parametrize("kind", [M.ROT_PAIRWISE, M.ROT_HALF])
def test_large_angles(kind):
    """Positions times one radian, up to and past where the angle reduction hands over to the library's."""
    t = _make(1, 64, 1, 2, 2, 16, kind, 8, F32, seed=5)
    t["rot"] = torch.logspace(0, 6, 64, device=DEV).view(1, 64, 1, 1) * torch.linspace(-1.0, 1.0, 8, device=DEV)
    t["rot"] = t["rot"].expand(1, 64, 2, 8).contiguous()
    _all(t, 2, kind)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_without_bias_and_many_tokens(dtype):
    """Several workgroups share the sums over tokens."""
    _all(_make(3, 1500, 2, 4, 2, 64, M.ROT_QUAT, 4, dtype, bias=False, seed=6), 4, M.ROT_QUAT)


def test_gradient_against_differences():
    t = _make(1, 5, 2, 4, 2, 16, M.ROT_QUAT, 2, F32, seed=7)
    _, got = _all(t, 4, M.ROT_QUAT)
    o = {k: _np(v) for k, v in t.items()}
    rng = np.random.default_rng(3)

    def loss(a):
        return sum((qk_norm.qk_fwd(a[n], a["w" + n], a["b" + n], a["rot"], M.ROT_QUAT, 4, EPS)
                    * o["d_%shat" % n]).sum() for n in ("q", "k"))

    for k in ("q", "k", "wq", "wk", "bq", "bk", "rot"):
        v = rng.standard_normal(o[k].shape)
        num = (loss({**o, k: o[k] + 1e-6 * v}) - loss({**o, k: o[k] - 1e-6 * v})) / 2e-6
        g = _np(got["d_" + k])
        assert abs((g * v).sum() - num) <= TOL[F32] * np.linalg.norm(g) * np.linalg.norm(v) + 1e-7 * abs(num), k


def test_nothing_to_do_wanted_only_and_streams():
    t = _make(2, 40, 1, 4, 2, 32, M.ROT_HALF, 8, BF16, rot_h=1, seed=8)
    args = [t[n] for n in ("q", "k", "wq", "wk", "bq", "bk", "rot")]
    d = M.qk_desc(t["q"], t["k"], 4, M.ROT_HALF, rot=t["rot"], eps=EPS)
    full = M.moments_qk_bwd(d, *args, t["d_qhat"], t["d_khat"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for k in ("q", "k", "wq", "wk", "bq", "bk", "rot"):
            one = M.moments_qk_bwd(d, *args, t["d_qhat"], t["d_khat"], want=(k,))
            assert torch.equal(one["d_" + k], full["d_" + k])
            assert all(v is None for n, v in one.items() if n != "d_" + k)
    st.synchronize()
    e = [t["q"][:, :0], t["k"][:, :0], *args[2:6], t["rot"][:, :0]]
    d = M.qk_desc(e[0], e[1], 4, M.ROT_HALF, rot=e[6], eps=EPS)
    qh, _ = M.moments_qk_fwd(d, *e)
    assert qh.shape == (2, 0, 1, 4, 32)
    g = M.moments_qk_bwd(d, *e, t["d_qhat"][:, :0], t["d_khat"][:, :0])
    assert torch.count_nonzero(g["d_wq"]) == 0 and torch.count_nonzero(g["d_bk"]) == 0


def test_offsets_past_32_bits():
    """Rows cut out of a projection of more than 2^31 values."""
    s, width = 70_000, 32_768
    wide = torch.zeros(1, s, width, dtype=BF16, device=DEV)
    t = _make(1, 3, 1, 4, 2, 64, M.ROT_PAIRWISE, 8, BF16, seed=9)
    assert wide.numel() > 2 ** 31
    wide[:, -3:, :128] = t["q"].reshape(1, 3, 128)
    q = wide[:, :, :128].view(1, s, 1, 2, 64)
    rot = torch.zeros(1, s, 4, 8, dtype=BF16, device=DEV)
    rot[:, -3:] = t["rot"]
    d = M.qk_desc(q, q, 4, M.ROT_PAIRWISE, rot=rot, eps=EPS)
    qh, _ = M.moments_qk_fwd(d, q, q, t["wq"], t["wk"], t["bq"], t["bk"], rot)
    ref = qk_norm.qk_fwd(_np(t["q"]), _np(t["wq"]), _np(t["bq"]), _np(t["rot"]), M.ROT_PAIRWISE, 4, EPS)
    _check("qhat", qh[:, -3:], ref, TOL[BF16])
