"""The norms with rotation where their arithmetic ends: no eps, subnormal mean squares,
large angles, empty batches, rows cut out of a projection at any element.

Tolerances are those of test_gpu_qk.py unless a test states its own."""
import ctypes

import numpy as np
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from mamba_ssm_chunkwise_amd import _lib
from oracle import qk_norm
from test_gpu_qk import BF16, DEV, F32, KINDS, TOL, _check, _make, _np

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "wq", "wk", "bq", "bk", "rot")


def _run(t, h, kind, eps, out=None):
    d = M.qk_desc(t["q"], t["k"], h, kind, rot=t["rot"], eps=eps)
    args = [t[n] for n in NAMES]
    return M.moments_qk_fwd(d, *args), M.moments_qk_bwd(d, *args, t["d_qhat"], t["d_khat"], out=out)


def _against_oracle(t, h, kind, eps):
    hats, got = _run(t, h, kind, eps)
    o = {k: _np(v) for k, v in t.items()}
    for i, n in enumerate(("q", "k")):
        a = (o[n], o["w" + n], o["b" + n], o["rot"], kind, h, eps)
        _check(n + "hat", hats[i], qk_norm.qk_fwd(*a), TOL[t["q"].dtype])
        d_x, d_w, d_b, _ = qk_norm.qk_bwd(*a, o["d_%shat" % n])
        _check("d_" + n, got["d_" + n], d_x, TOL[t["q"].dtype])
        _check("d_w" + n, got["d_w" + n], d_w, TOL[F32])
        _check("d_b" + n, got["d_b" + n], d_b, TOL[F32])
    return hats, got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind,width", KINDS)
@pytest.mark.parametrize("c,h,g,r", [(1, 3, 3, 24), (2, 2, 2, 128), (1, 4, 2, 24), (3, 1, 1, 30), (1, 24, 2, 45)])
def test_without_eps(dtype, kind, width, c, h, g, r):
    """Nine tokens never fill the places that a wave has for tokens."""
    if kind == M.ROT_HALF and r % 2:
        pytest.skip("half-split rows are even")
    print(f"[case] eps=0 kind={kind} c={c} h={h} g={g} r={r} {dtype}", flush=True)
    _against_oracle(_make(1, 9, c, h, g, r, kind, width, dtype, seed=r), h, kind, 0.0)


def test_gradients_of_no_tokens_need_no_weights():
    """The C call with s = 0 and every input NULL: the parameters' gradients are zero."""
    h, r = 4, 24
    d = M.QkDesc(2, 0, 1, h, 2, r, 0, 0, 8, 0, h, _lib.F32, M.ROT_PAIRWISE, 1e-5)
    ws = torch.empty(M.moments_qk_workspace_size(d), dtype=torch.uint8, device=DEV)
    d_w = [torch.full((r,), float("nan"), device=DEV) for _ in range(2)]
    rc = _lib.load().moments_qk_bwd(ctypes.byref(d), *[None] * 11, d_w[0].data_ptr(), d_w[1].data_ptr(), None, None,
                                    None, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and all(torch.count_nonzero(v) == 0 for v in d_w)


def _poisoned(t, h):
    """Gradients to be written over: each holds NaN."""
    return {"d_" + n: torch.full_like(t[n], float("nan")) for n in NAMES if t[n] is not None}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rot_h", [1, None])
@pytest.mark.parametrize("b,s,h", [(0, 5, 4), (2, 0, 4), (2, 5, 0)])
def test_gradients_of_empty_inputs(dtype, rot_h, b, s, h):
    """No sequences, no tokens, no heads: what is left of the gradients is zero."""
    t = _make(b, s, 2, h, 2, 24, M.ROT_PAIRWISE, 4, dtype, rot_h=rot_h, seed=1)
    _, got = _run(t, h, M.ROT_PAIRWISE, 1e-5, out=_poisoned(t, h))
    torch.cuda.synchronize()
    for k, v in got.items():
        assert torch.equal(v, torch.zeros_like(v)), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r", [24, 45])
def test_rows_of_zeros_under_a_subnormal_eps(dtype, r):
    """Their mean square plus eps is subnormal: 1 / sqrt is 2^65, and the rows' norm is zero, not NaN."""
    t = _make(1, 10, 1, 2, 2, r, M.ROT_PAIRWISE, 4, dtype, seed=3)
    for n in ("q", "k"):
        t[n][:, ::2] = 0.0
    hats, got = _against_oracle(t, 2, M.ROT_PAIRWISE, 2.0 ** -130)
    o = {k: _np(v) for k, v in t.items()}
    for n in ("q", "k"):      # the other rows' gradients, which are 2^65 times smaller
        d_x = qk_norm.qk_bwd(o[n], o["w" + n], o["b" + n], o["rot"], M.ROT_PAIRWISE, 2, 2.0 ** -130,
                             o["d_%shat" % n])[0]
        _check("d_" + n, got["d_" + n][:, 1::2], d_x[:, 1::2], TOL[dtype])


def test_angles_next_to_multiples_of_a_right_angle():
    """float32 angles next to k pi/2 up to 1e5: the sine or cosine is tiny, and is right to its own last bits.

    The rows are (1, 0), so that hat is (cos, sin) times 1 up to a dozen roundings of 2^-24: 2^-20 bounds them."""
    x = (np.arange(1, 63000) * (np.pi / 2)).astype(np.float32)
    n = x.size
    q = torch.zeros(1, n, 1, 1, 2, device=DEV)
    q[..., 0] = 1.0
    w = torch.full((2,), 0.5 ** 0.5, device=DEV)
    rot = torch.from_numpy(x).to(DEV).view(1, n, 1, 1)
    hat, _ = M.moments_qk_fwd(M.qk_desc(q, q, 1, M.ROT_PAIRWISE, rot=rot, eps=0.0), q, q, w, w, rot=rot)
    got = _np(hat)[0, :, 0, 0]
    ref = np.stack([np.cos(x.astype(np.float64)), np.sin(x.astype(np.float64))], -1)
    err = np.abs(got - ref) / np.abs(ref)
    print(f"[compare] relative error of the smallest values: {err.max():.2e}", flush=True)
    assert err.max() <= 2.0 ** -20


@pytest.mark.parametrize("kind", [M.ROT_PAIRWISE, M.ROT_HALF])
def test_large_angles_in_bf16(kind):
    """Both of the reductions that bf16 rows use: below 1e5 and from there on."""
    t = _make(1, 64, 1, 2, 2, 16, kind, 8, BF16, seed=5)
    rot = torch.logspace(0, 6, 64, device=DEV).view(1, 64, 1, 1) * torch.linspace(-1.0, 1.0, 8, device=DEV)
    t["rot"] = rot.expand(1, 64, 2, 8).to(BF16).contiguous()
    assert (t["rot"].abs() > 1e5).any() and (t["rot"].abs() < 1e5).any()
    _against_oracle(t, 2, kind, 1e-5)


def test_bias_gradients_of_very_many_heads():
    """2^26 of them: more columns than one launch of the sums has threads for. One token, no rotation:
    each bias gradient is its cotangent."""
    g, h, r = 8192, 524_288, 128
    x = torch.randn(1, 1, 1, g, r, device=DEV).to(BF16)
    w, bias = torch.ones(r, device=DEV), torch.zeros(h, r, device=DEV)
    d_q, d_k = (torch.randn(1, 1, 1, h, r, device=DEV).to(BF16) for _ in range(2))
    d = M.qk_desc(x, x, h, M.ROT_NONE)
    got = M.moments_qk_bwd(d, x, x, w, w, bias, bias, None, d_q, d_k, want=("wq", "bq", "bk"))
    assert torch.equal(got["d_bq"], d_q.float().view(h, r)) and torch.equal(got["d_bk"], d_k.float().view(h, r))
    n = x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-5).sqrt()
    ref = (n * d_q.double().view(1, 1, 1, g, h // g, r).sum(4)).sum((0, 1, 2, 3))
    _check("d_wq", got["d_wq"], _np(ref), TOL[F32])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r,at", [(45, (0, 45)), (24, (3, 29)), (128, (1, 130)), (16, (8, 25))])
def test_columns_that_start_at_any_element(dtype, r, at):
    """Queries and keys cut out of one projection: the base need not be aligned either."""
    t = _make(2, 9, 1, 2, 1, r, M.ROT_PAIRWISE, 4, dtype, seed=r)
    wide = torch.randn(2, 9, at[1] + r + 3, device=DEV).to(dtype)
    for n, lo in zip(("q", "k"), at):
        t[n] = wide[:, :, lo:lo + r].view(2, 9, 1, 1, r)
    print(f"[case] r={r} at={at} {dtype}: {t['q'].data_ptr() % 16} {t['k'].data_ptr() % 16}", flush=True)
    hats, got = _against_oracle(t, 2, M.ROT_PAIRWISE, 1e-5)
    own = dict(t, q=t["q"].contiguous(), k=t["k"].contiguous())      # aligned rows of their own
    hats2, got2 = _run(own, 2, M.ROT_PAIRWISE, 1e-5)
    for a, b in zip(hats, hats2):
        _check("hat", a, _np(b), TOL[dtype])


def test_finite_check_of_the_forward(monkeypatch):
    t = _make(1, 7, 1, 2, 2, 24, M.ROT_PAIRWISE, 4, F32, seed=2)
    d = M.qk_desc(t["q"], t["k"], 2, M.ROT_PAIRWISE, rot=t["rot"])
    args = [t[n] for n in NAMES]
    monkeypatch.setenv("MOMENTS_CHECK_FINITE", "1")
    M.moments_qk_fwd(d, *args)
    t["k"][0, 3, 0, 1, 5] = float("inf")
    with pytest.raises(M.MomentsError) as e:
        M.moments_qk_fwd(d, *args)
    assert e.value.code == _lib.ENONFINITE
