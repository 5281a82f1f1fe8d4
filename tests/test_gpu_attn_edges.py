"""Linear attention at its edges: values that are not finite, cleared states, buffers
that a caller uses twice, empty inputs, the finite check of single tokens.

Tolerances are those of test_gpu_attn.py."""
import numpy as np
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from mamba_ssm_chunkwise_amd import _lib
from oracle import attn_seq
from test_gpu_attn import BF16, DEV, F32, TOL, _check, _make, _np

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
INPUTS = ("xhat", "bhat", "qhat", "da")


def _args(t):
    return [t[n] for n in INPUTS]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,s,h,p,lens", [(2, 50, 3, 24, None), (1, 2300, 2, 96, None), (4, 2300, 2, 32, [5, 2300, 0, 900])])
def test_states_written_over_the_ones_that_were_read(dtype, b, s, h, p, lens):
    """h_last on h0, and d_h0 on d_h_last: one segment, several, and lengths that leave segments empty."""
    print(f"[case] in place b={b} s={s} {dtype}", flush=True)
    t = _make(b, s, 1, h, 1, p, 40, dtype, seed=b + s)
    a = _args(t)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    d = M.attn_desc(a[0], a[1], valid_lens=n)
    y, last, saved = M.moments_attn_fwd_save(d, *a, t["h0"])
    g = M.moments_attn_bwd_saved(d, *a, t["h0"], saved, t["d_y"], t["d_last"])
    for save in (False, True):
        h0 = t["h0"].clone()
        if save:
            y2, last2, saved2 = M.moments_attn_fwd_save(d, *a, h0, h_last=h0)
        else:
            y2, last2 = M.moments_attn_fwd(d, *a, h0, h_last=h0)
        assert last2 is h0 and torch.equal(y, y2) and torch.equal(last, h0)
    for save in (False, True):
        dl = t["d_last"].clone()
        if save:
            g2 = M.moments_attn_bwd_saved(d, *a, t["h0"], saved2, t["d_y"], dl, out={"d_h0": dl})
        else:
            g2 = M.moments_attn_bwd(d, *a, t["h0"], t["d_y"], dl, out={"d_h0": dl})
        for k in g:
            assert torch.equal(g[k], g2[k]), k


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_without_heads(dtype):
    """h = 0: keys and queries still have gradients, and they are zero."""
    t = _make(2, 5, 1, 1, 1, 4, 8, dtype, seed=1)
    k, q = (torch.randn(2, 5, 1, 2, 8, device=DEV).to(dtype) for _ in range(2))
    x, da = t["xhat"][:, :, :, :0].contiguous(), t["da"][:, :, :0].contiguous()
    d = M.attn_desc(x, k)
    out = {"d_bhat": torch.full_like(k, NAN), "d_qhat": torch.full_like(q, NAN)}
    got = M.moments_attn_bwd(d, x, k, q, da, None, x, out=out)
    torch.cuda.synchronize()
    for n in ("d_bhat", "d_qhat"):
        assert torch.equal(got[n], torch.zeros_like(k)), n


def test_the_largest_launches():
    """As many chains as a launch holds: forwards and single tokens 2^24 - 1, gradients 2^23 - 1."""
    n = 2 ** 24 - 1
    one = lambda *shape: torch.ones(n, *shape, device=DEV)  # noqa: E731
    x, k, da = one(1, 1, 1, 1), one(1, 1, 1, 1), torch.zeros(n, 1, 1, device=DEV)
    h0 = torch.arange(n, dtype=torch.float32, device=DEV).view(n, 1, 1, 1) % 1024
    d = M.attn_desc(x, k)
    y, last = M.moments_attn_fwd(d, x, k, k, da, h0)
    assert torch.equal(last, h0 + 1) and torch.equal(y.view(-1), last.view(-1))
    assert torch.equal(M.moments_attn_step(d, x, k, k, da, last).view(-1), h0.view(-1) + 2)
    n = 2 ** 23 - 1
    x, k, da, h0 = x[:n, :0], k[:n, :0], da[:n, :0], h0[:n].contiguous()
    got = M.moments_attn_bwd(M.attn_desc(x, k), x, k, k, da, h0, x, h0)
    assert torch.equal(got["d_h0"], h0)


def test_finite_check_of_single_tokens(monkeypatch):
    t = _make(3, 1, 1, 2, 2, 16, 16, BF16, seed=2)
    a = _args(t)
    d = M.attn_desc(a[0], a[1])
    pool = torch.full((4, 2, 16, 16), NAN, device=DEV)      # a slot that no sequence has is not looked at
    pool[:2] = 0.0
    slots = torch.tensor([1, -1, 0], dtype=torch.int32, device=DEV)
    monkeypatch.setenv("MOMENTS_CHECK_FINITE", "1")
    M.moments_attn_step(d, *a, pool, slots)
    pool[0, 1, 3, 5] = INF
    with pytest.raises(M.MomentsError) as e:
        M.moments_attn_step(d, *a, pool, slots)
    assert e.value.code == _lib.ENONFINITE


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,h,g,p,r", [(1, 2, 1, 16, 24), (3, 2, 2, 70, 45), (2, 1, 1, 130, 128)])
def test_single_tokens_start_anew_on_a_slot_that_holds_anything(dtype, c, h, g, p, r):
    """da = -inf (or the type's lowest value): the slot's NaN and infinities are gone."""
    t = _make(3, 1, c, h, g, p, r, dtype, seed=p)
    t["da"][0], t["da"][1], t["da"][2] = -INF, torch.finfo(dtype).min, -0.5
    a = _args(t)
    pool = torch.full((3, h, p, r), NAN, device=DEV)
    pool[1] = INF
    pool[2] = 0.25
    ref = pool.clone()
    ref[:2] = 0.0
    y = M.moments_attn_step(M.attn_desc(a[0], a[1]), *a, pool)
    o = [_np(v) for v in a]
    o[3] = np.maximum(o[3], -1e4)
    ry, rs = attn_seq.attn_fwd(*o, _np(ref))
    _check("y", y, ry, TOL[dtype])
    _check("state", pool, rs, TOL[F32])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_cleared_state_is_gone_however_much_later_decays_grow(dtype):
    """A state of 1e30, cleared, then log-decays of +1 on zero values: nothing comes back."""
    t = _make(1, 2200, 1, 1, 1, 16, 24, dtype, seed=8)
    t["xhat"].zero_()
    t["h0"][:] = 1e30
    t["da"].zero_()
    t["da"][:, 3:70] = 1.0
    t["da"][:, 1] = -INF
    a = _args(t)
    y, last = M.moments_attn_fwd(M.attn_desc(a[0], a[1]), *a, t["h0"])
    assert torch.count_nonzero(y[:, 1:]) == 0 and torch.count_nonzero(last) == 0
    assert torch.count_nonzero(y[:, 0]) > 0


def _cleared(t, cut, dtype):
    """The oracle's outputs of what follows token `cut`, where the state is cleared."""
    tail = [v[:, cut:].contiguous() for v in _args(t)]
    o = [_np(v) for v in tail]
    o[3] = np.maximum(o[3], -1e4)
    return attn_seq.attn_fwd(*o, None)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,p,r,s,cut", [(1, 32, 40, 150, 0), (1, 32, 40, 150, 77), (3, 24, 32, 60, 25),
                                         (1, 37, 45, 90, 64), (2, 128, 128, 70, 33), (1, 64, 128, 2300, 1111)])
@pytest.mark.parametrize("bad", ["h0", "xhat", "bhat", "qhat", "da", "inf xhat", "inf bhat"])
def test_a_cleared_state_forgets_what_is_not_finite(dtype, c, p, r, s, cut, bad):
    """da = -inf starts the sequence anew, also behind a NaN or an infinity, in its chunk or an earlier one."""
    print(f"[case] {bad} c={c} p={p} r={r} s={s} cut={cut} {dtype}", flush=True)
    t = _make(1, s, c, 2, 1, p, r, dtype, seed=s + cut)
    name, v = bad.split()[-1], INF if " " in bad else NAN
    if name != "h0" and cut == 0:
        pytest.skip("nothing is before the first token")
    if name == "h0":
        t["h0"][:] = NAN
    else:
        t[name][:, max(0, cut - 5)] = v
    t["da"][:, cut] = -INF
    a = _args(t)
    y, last, saved = M.moments_attn_fwd_save(M.attn_desc(a[0], a[1]), *a, t["h0"])
    ry, rl = _cleared(t, cut, dtype)
    _check("y", y[:, cut:], ry, TOL[dtype])
    _check("h_last", last, rl, TOL[F32])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,p,r,at", [(1, 32, 40, 40), (3, 24, 32, 15), (1, 37, 45, 10), (2, 128, 128, 29),
                                      (4, 70, 64, 3)])
@pytest.mark.parametrize("name", ["xhat", "bhat", "qhat", "da"])
@pytest.mark.parametrize("v", [NAN, INF, -INF])
def test_later_tokens_do_not_reach_earlier_ones(dtype, c, p, r, at, name, v):
    """A NaN or an infinity at a token: the outputs before it are what they are without it."""
    if name == "da" and v == -INF:
        pytest.skip("a cleared state")
    print(f"[case] {name} {v} c={c} p={p} r={r} at={at} {dtype}", flush=True)
    t = _make(1, at + 50, c, 2, 2, p, r, dtype, seed=at)
    a = _args(t)
    d = M.attn_desc(a[0], a[1])
    clean = [v_.clone() for v_ in a]
    t[name][:, at] = v
    y, _ = M.moments_attn_fwd(d, *a, t["h0"])
    o = [_np(x[:, :at]) for x in clean]
    ry, _ = attn_seq.attn_fwd(*o, _np(t["h0"]))
    _check("y", y[:, :at], ry, TOL[dtype])
    # and from there on it is seen: no output that reads the value is finite (a NaN or an infinite
    # query is seen by its own token alone)
    seen = y[:, at] if name == "qhat" else y[:, at:]
    assert not torch.isfinite(seen).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_bad_value_stays_in_its_state_row(dtype):
    """x[t, 0, 0, 7] = NaN reaches y[t:, :, 0, 7] and the state's row 7, nothing else."""
    t = _make(1, 100, 1, 2, 1, 72, 64, dtype, seed=7)
    a = _args(t)
    d = M.attn_desc(a[0], a[1])
    clean, last0 = M.moments_attn_fwd(d, *a, t["h0"])
    a[0][0, 50, 0, 0, 7] = NAN
    y, last = M.moments_attn_fwd(d, *a, t["h0"])
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[:, 50:, :, 0, 7] = True
    assert torch.isnan(y[hit]).all() and torch.isfinite(y[~hit]).all()
    _check("y", torch.where(hit, 0.0, y.float()), _np(torch.where(hit, 0.0, clean.float())), 2 * TOL[dtype])
    hit = torch.zeros_like(last, dtype=torch.bool)
    hit[:, 0, 7] = True
    assert torch.isnan(last[hit]).all()
    _check("h_last", torch.where(hit, 0.0, last), _np(torch.where(hit, 0.0, last0)), 2 * TOL[F32])


def test_autograd_sees_what_is_written_in_place():
    """A tensor that a graph holds for its backward, then given as the state or as an output."""
    t = _make(2, 1, 1, 2, 2, 16, 24, F32, seed=9)
    a = _args(t)
    d = M.attn_desc(a[0], a[1])

    def held(v):
        leaf = torch.randn_like(v).requires_grad_()
        return leaf.exp()            # its backward reads the result

    for write in (lambda v: M.moments_attn_step(d, *a, v), lambda v: M.moments_attn_fwd(d, *a, t["h0"], h_last=v),
                  lambda v: M.moments_attn_fwd(d, *a, v, h_last=v),
                  lambda v: M.moments_attn_bwd(d, *a, t["h0"], t["d_y"], out={"d_h0": v})):
        v = held(t["h0"])
        write(v.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            v.sum().backward()
    v = held(t["h0"])
    M.moments_attn_fwd(d, *a, v.detach())          # read only
    v.sum().backward()


def _beside_rounding(name, got, ref):
    """The error of a bf16 result, at most 1.1 times that of rounding the exact one: scores of 17 bits add
    2^-17 of their terms to its 2^-9."""
    alone = torch.from_numpy(ref).to(BF16).double().numpy()
    e, e0 = np.linalg.norm(_np(got) - ref), np.linalg.norm(alone - ref)
    print(f"[compare] {name}: {e:.3e}, the rounding's alone {e0:.3e}", flush=True)
    assert e <= 1.1 * e0, (name, e, e0)


@pytest.mark.parametrize("s,c,h,g,p,r", [(1, 1, 8, 8, 64, 128), (2, 2, 4, 2, 37, 45), (7, 3, 4, 4, 64, 64), (16, 4, 2, 1, 128, 128),
                                         (64, 1, 2, 2, 64, 128), (21, 3, 2, 1, 96, 24)])
def test_bf16_outputs_are_right_to_their_rounding(s, c, h, g, p, r):
    """Within one chunk from a state of zeros, where nothing but the scores is rounded on the way."""
    t = _make(3, s, c, h, g, p, r, BF16, seed=s + p, h0=False)
    a = _args(t)
    y, _ = M.moments_attn_fwd(M.attn_desc(a[0], a[1]), *a)
    _beside_rounding("y", y, attn_seq.attn_fwd(*[_np(v) for v in a])[0])


@pytest.mark.parametrize("s,c,h,g,p,r", [(1, 1, 8, 8, 64, 128), (2, 2, 4, 2, 37, 45), (7, 3, 4, 4, 64, 64), (16, 4, 2, 1, 128, 128),
                                         (64, 1, 2, 2, 64, 128), (21, 3, 2, 1, 96, 24)])
def test_bf16_gradients_are_right_to_their_rounding(s, c, h, g, p, r):
    """Likewise, with no cotangent of the last state. (d_xhat of the widest shapes has scores of one piece.)"""
    t = _make(3, s, c, h, g, p, r, BF16, seed=s + p, h0=False)
    a = _args(t)
    got = M.moments_attn_bwd(M.attn_desc(a[0], a[1]), *a, None, t["d_y"])
    ref = attn_seq.attn_bwd(*[_np(v) for v in a], None, _np(t["d_y"]))
    for k in ("d_xhat", "d_bhat", "d_qhat", "d_da"):
        if k != "d_xhat" or p <= 64 or r <= 64:
            _beside_rounding(k, got[k], ref[k])
