"""GPU parity of linear attention with a decay for each head (chunked forward,
gradients, single tokens) with the 64-bit recurrence of oracle/attn_seq.py.

Tolerances. float32: products and sums in fp32, at most a few hundred terms of unit
roundoff 2^-24 each: 1e-5 bounds them (normwise, and elementwise over the largest
magnitude). bfloat16: the result, the scores and the copy of the state are each
rounded once (at most 2^-9 of a term): 3 * 2^-9 normwise; elementwise, over the largest
magnitude, the same. Float32 states of bfloat16 inputs are held to the float32 bound.
"""
import numpy as np
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from oracle import attn_seq
from parity_util import max_err, rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {torch.float32: 1e-5, torch.bfloat16: 3 * 2.0 ** -9}


def _np(x):
    return None if x is None else x.detach().double().cpu().numpy()


def _make(b, s, c, h, g, p, r, dtype, seed=1, h0=True, resets=False):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    f = lambda *shape: torch.randn(*shape, device=DEV, generator=gen)  # noqa: E731
    t = {"xhat": f(b, s, c, h, p).to(dtype), "bhat": f(b, s, c, g, r).to(dtype),
         "qhat": (f(b, s, c, g, r) * r ** -0.5).to(dtype)}
    da = -torch.nn.functional.softplus(f(b, s, h) - 1.0)
    if resets:
        da[torch.rand(b, s, h, device=DEV, generator=gen) < 0.04] = -float("inf")
        da[torch.rand(b, s, h, device=DEV, generator=gen) < 0.02] = torch.finfo(dtype).min
    t["da"] = da.to(dtype)
    t["h0"] = f(b, h, p, r) * 0.5 if h0 else None
    t["d_y"], t["d_last"] = f(b, s, c, h, p).to(dtype), f(b, h, p, r) * 0.1
    return t


def _check(name, got, ref, tol):
    got = _np(got)
    assert np.all(np.isfinite(got)), f"{name}: non-finite values"
    e, m = rel_err(got, ref), max_err(got, ref)
    print(f"[compare] {name}: normwise {e:.2e} max-elementwise {m:.2e}", flush=True)
    assert e <= tol and m <= tol, f"{name}: {e:.2e}/{m:.2e} above {tol:.1e}"


def _all(t, lens=None, valid=None, backward=True, oracle=None):
    """Forward and gradients against the oracle; returns the GPU outputs."""
    dt = t["xhat"].dtype
    s = t["xhat"].shape[1]
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    d = M.attn_desc(t["xhat"], t["bhat"], valid_len=valid, valid_lens=dl)
    a = (t["xhat"], t["bhat"], t["qhat"], t["da"], t["h0"])
    y, last, saved = M.moments_attn_fwd_save(d, *a)
    top = s if valid is None else min(valid, s)
    n = np.full(t["xhat"].shape[0], top) if lens is None else np.clip(lens, 0, top)
    live = np.arange(s)[None] < n[:, None]
    o = {k: _np(v) for k, v in (oracle or t).items()}
    for k in ("xhat", "bhat", "qhat", "da", "d_y"):     # the oracle stops at the length; its sums need finite rows
        o[k] = np.where(live.reshape(live.shape + (1,) * (o[k].ndim - 2)), o[k], 0.0)
    o["da"] = np.maximum(o["da"], -1e4)
    ry, rl = attn_seq.attn_fwd(o["xhat"], o["bhat"], o["qhat"], o["da"], o["h0"], n)
    _check("y", y, ry, TOL[dt])
    _check("h_last", last, rl, TOL[torch.float32])
    assert np.all(_np(y)[~live] == 0)
    out = {"y": y, "h_last": last}
    if backward:
        ref = attn_seq.attn_bwd(o["xhat"], o["bhat"], o["qhat"], o["da"], o["h0"], o["d_y"], o["d_last"], n)
        got = M.moments_attn_bwd_saved(d, *a, saved, t["d_y"], t["d_last"])
        for k, v in got.items():
            if v is None:
                assert k == "d_h0" and t["h0"] is None
                continue
            _check(k, v, ref[k], TOL[v.dtype])
            if k != "d_h0":
                assert np.all(_np(v)[~live] == 0), f"{k} is not zero past the length"
        again = M.moments_attn_bwd(d, *a, t["d_y"], t["d_last"])      # makes the saved states itself
        for k, v in got.items():
            assert v is None or torch.equal(v, again[k]), k
        out.update(got)
    torch.cuda.synchronize()
    return out


F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("s", [1, 2, 31, 32, 33, 63, 64, 65, 130])
def test_lengths(dtype, s):
    print(f"[case] s={s} {dtype}", flush=True)
    _all(_make(2, s, 1, 3, 3, 24, 40, dtype, seed=s))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,s", [(2, 33), (2, 64), (3, 21), (3, 22), (3, 50), (4, 16), (4, 17), (4, 40)])
def test_channels(dtype, c, s):
    """Rows of one token see each other; with three channels a token straddles tiles of 16 rows."""
    print(f"[case] c={c} s={s} {dtype}", flush=True)
    _all(_make(2, s, c, 2, 2, 16, 32, dtype, seed=10 * c + s))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p,r", [(1, 1), (3, 5), (8, 8), (16, 128), (37, 45), (64, 64), (64, 128), (65, 66), (96, 100),
                                 (128, 64), (128, 128), (136, 128), (200, 20)])
def test_state_shapes(dtype, p, r):
    """Odd and unaligned rows, and state rows in one or several workgroups' tiles."""
    print(f"[case] p={p} r={r} {dtype}", flush=True)
    _all(_make(1, 70, 1, 2, 2, p, r, dtype, seed=p + r))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("h,g", [(1, 1), (4, 1), (6, 2), (6, 3), (12, 4)])
def test_shared_keys(dtype, h, g):
    print(f"[case] h={h} g={g} {dtype}", flush=True)
    _all(_make(2, 75, 2, h, g, 20, 24, dtype, seed=h + g))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("h0", [False, True])
def test_ragged_lengths_with_garbage_past_them(dtype, h0):
    """Lengths of zero, one, a chunk, and past valid_len; NaN and infinities where nothing is to be read."""
    lens = [0, 1, 64, 65, 200, 90]
    t = _make(6, 100, 1, 2, 1, 16, 24, dtype, seed=3, h0=h0)
    live = torch.arange(100, device=DEV)[None] < torch.tensor(lens, device=DEV).clamp(max=95)[:, None]
    for k, bad in (("xhat", float("nan")), ("bhat", float("inf")), ("qhat", float("nan")), ("da", float("nan")),
                   ("d_y", -float("inf"))):
        t[k][~live] = bad
    _all(t, lens=lens, valid=95)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1, 3])
def test_cleared_states(dtype, c):
    """da of -inf or of the type's lowest value: a decay of zero, also several in one chunk."""
    _all(_make(2, 150, c, 2, 2, 16, 32, dtype, seed=4, resets=True))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weak_and_growing_decays(dtype):
    """No decay at all (the state only grows), and positive log-decays."""
    t = _make(1, 200, 1, 2, 2, 16, 32, dtype, seed=5)
    t["da"].zero_()
    _all(t)
    t["da"].fill_(0.015625)
    _all(t)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,g,p", [(1, 2, 32), (2, 1, 32), (4, 2, 96)])
def test_few_long_chains(dtype, c, g, p):
    """Few chains: the walks are split into segments, forwards and backwards."""
    print(f"[case] segments c={c} g={g} {dtype}", flush=True)
    _all(_make(1, 2300 // c, c, 2, g, p, 40, dtype, seed=6), lens=[2101 // c])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_against_differences(dtype):
    """Central differences of the 64-bit forward along random directions, at the GPU's gradients."""
    t = _make(1, 70, 2, 2, 1, 16, 24, dtype, seed=8)
    got = _all(t)
    rng = np.random.default_rng(1)
    o = {k: _np(v) for k, v in t.items()}
    names = {"xhat": "d_xhat", "bhat": "d_bhat", "qhat": "d_qhat", "da": "d_da", "h0": "d_h0"}

    def loss(e, k, v):
        a = {n: o[n] + (e * v if n == k else 0.0) for n in names}
        y, last = attn_seq.attn_fwd(a["xhat"], a["bhat"], a["qhat"], a["da"], a["h0"])
        return (y * o["d_y"]).sum() + (last * o["d_last"]).sum()

    for k, key in names.items():
        v = rng.standard_normal(o[k].shape)
        num = (loss(1e-5, k, v) - loss(-1e-5, k, v)) / 2e-5
        g = _np(got[key])
        tol = TOL[got[key].dtype] * np.linalg.norm(g) * np.linalg.norm(v) / np.sqrt(g.size) * 8 + 1e-6 * abs(num)
        assert abs((g * v).sum() - num) <= tol, (k, (g * v).sum(), num)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pieces_and_single_tokens_continue_a_sequence(dtype):
    """A prompt in two pieces, then token by token, against the whole sequence."""
    t = _make(3, 90, 2, 4, 2, 32, 48, dtype, seed=9)
    a = [t[k] for k in ("xhat", "bhat", "qhat", "da")]
    whole, last = M.moments_attn_fwd(M.attn_desc(a[0], a[1]), *a, t["h0"])
    state, ys = t["h0"], []
    for lo, hi in ((0, 33), (33, 80)):
        part = [x[:, lo:hi].contiguous() for x in a]
        y, state = M.moments_attn_fwd(M.attn_desc(part[0], part[1]), *part, state)
        ys.append(y)
    pool = torch.full((5, 4, 32, 48), float("nan"), device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    pool[slots.long()] = state
    for i in range(80, 90):
        part = [x[:, i:i + 1].contiguous() for x in a]
        ys.append(M.moments_attn_step(M.attn_desc(part[0], part[1]), *part, pool, slots))
    _check("y", torch.cat(ys, 1), _np(whole), 2 * TOL[dtype])
    _check("state", pool[slots.long()], _np(last), 2 * TOL[torch.float32])
    assert torch.isnan(pool[[1, 3]]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,h,g,p,r", [(1, 1, 1, 1, 1), (2, 4, 2, 7, 9), (3, 2, 1, 33, 32), (4, 3, 3, 64, 64),
                                       (1, 8, 1, 100, 99), (2, 2, 2, 130, 128)])
def test_single_tokens(dtype, c, h, g, p, r):
    print(f"[case] step c={c} h={h} p={p} r={r} {dtype}", flush=True)
    b, n = 5, 7
    t = _make(b, 1, c, h, g, p, r, dtype, seed=p + r)
    t["da"][1] = -float("inf")
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    pool = torch.randn(n, h, p, r, device=DEV, generator=gen)
    before = pool.clone()
    slots = torch.tensor([3, 6, -1, 0, 7], dtype=torch.int32, device=DEV)     # 7: outside the pool
    a = [t[k] for k in ("xhat", "bhat", "qhat", "da")]
    y = M.moments_attn_step(M.attn_desc(a[0], a[1]), *a, pool, slots)
    use = [0, 1, 3]
    o = [_np(x)[use] for x in a]
    o[3] = np.maximum(o[3], -1e4)
    ry, rs = attn_seq.attn_fwd(*o, _np(before)[[3, 6, 0]])
    _check("y", y[use], ry, TOL[dtype])
    _check("state", pool[[3, 6, 0]], rs, TOL[torch.float32])
    assert torch.count_nonzero(y[[2, 4]]) == 0 and torch.equal(pool[[1, 2, 4, 5]], before[[1, 2, 4, 5]])
    own = before[:b].clone()                                                  # no slots: sequence i in slot i
    y = M.moments_attn_step(M.attn_desc(a[0], a[1]), *a, own)
    o = [_np(x) for x in a]
    o[3] = np.maximum(o[3], -1e4)
    ry, rs = attn_seq.attn_fwd(*o, _np(before)[:b])
    _check("y", y, ry, TOL[dtype])
    _check("state", own, rs, TOL[torch.float32])


def test_nothing_to_do():
    z = lambda *shape: torch.zeros(*shape, device=DEV)  # noqa: E731
    h0 = torch.randn(2, 3, 4, 5, device=DEV)
    a = (z(2, 0, 1, 3, 4), z(2, 0, 1, 3, 5), z(2, 0, 1, 3, 5), z(2, 0, 3))
    d = M.attn_desc(a[0], a[1])
    y, last = M.moments_attn_fwd(d, *a, h0)
    assert y.numel() == 0 and torch.equal(last, h0)
    assert torch.equal(M.moments_attn_bwd(d, *a, h0, a[0], h0)["d_h0"], h0)
    a = (z(0, 7, 1, 3, 4), z(0, 7, 1, 3, 5), z(0, 7, 1, 3, 5), z(0, 7, 3))
    assert M.moments_attn_fwd(M.attn_desc(a[0], a[1]), *a)[0].shape == (0, 7, 1, 3, 4)


def test_wanted_gradients_only():
    t = _make(1, 70, 1, 4, 2, 16, 24, BF16, seed=12)
    a = [t[k] for k in ("xhat", "bhat", "qhat", "da", "h0")]
    d = M.attn_desc(a[0], a[1])
    full = M.moments_attn_bwd(d, *a, t["d_y"], t["d_last"])
    for k in ("xhat", "bhat", "qhat", "da", "h0"):
        one = M.moments_attn_bwd(d, *a, t["d_y"], t["d_last"], want=(k,))
        assert torch.equal(one["d_" + k], full["d_" + k])
        assert all(v is None for n, v in one.items() if n != "d_" + k)


def test_other_stream_and_repeats():
    """On a stream of its own, and the same bits each time."""
    t = _make(2, 300, 2, 4, 2, 64, 128, BF16, seed=13)
    a = [t[k] for k in ("xhat", "bhat", "qhat", "da", "h0")]
    d = M.attn_desc(a[0], a[1])
    y, last = M.moments_attn_fwd(d, *a)
    g = M.moments_attn_bwd(d, *a, t["d_y"], t["d_last"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y2, last2, saved = M.moments_attn_fwd_save(d, *a)
        g2 = M.moments_attn_bwd_saved(d, *a, saved, t["d_y"], t["d_last"])
    st.synchronize()
    assert torch.equal(y, y2) and torch.equal(last, last2)
    assert all(torch.equal(g[k], g2[k]) for k in g)


def test_graph_replays():
    """Captured once, replayed with new inputs, against the eager results."""
    t = _make(2, 200, 1, 4, 2, 64, 128, BF16, seed=14)
    a = [t[k] for k in ("xhat", "bhat", "qhat", "da", "h0")]
    d = M.attn_desc(a[0], a[1])
    fw = torch.empty(M.moments_attn_workspace_size(d, False), dtype=torch.uint8, device=DEV)
    bw = torch.empty(M.moments_attn_workspace_size(d, True), dtype=torch.uint8, device=DEV)

    def step():
        y, last, saved = M.moments_attn_fwd_save(d, *a, workspace=fw)
        return [y, last, *M.moments_attn_bwd_saved(d, *a, saved, t["d_y"], t["d_last"], workspace=bw).values()]

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        a[0].copy_(torch.randn_like(a[0]))
        a[3].copy_(-torch.rand_like(a[3]))
        graph.replay()
        torch.cuda.synchronize()
        for x, ref in zip(out, step()):
            assert torch.equal(x, ref)


def test_offsets_past_32_bits():
    """More than 2^31 values of x: the last tokens, behind a cleared state, against themselves alone."""
    s, tail, h, p = 140_000, 100, 128, 128
    x = torch.zeros(1, s, 1, h, p, dtype=BF16, device=DEV)
    k, q = torch.zeros(1, s, 1, 1, 16, dtype=BF16, device=DEV), torch.zeros(1, s, 1, 1, 16, dtype=BF16, device=DEV)
    da = torch.zeros(1, s, h, dtype=BF16, device=DEV)
    t = _make(1, tail, 1, h, 1, p, 16, BF16, seed=15, h0=False)
    t["da"][:, 0] = -float("inf")
    for big, key in ((x, "xhat"), (k, "bhat"), (q, "qhat"), (da, "da")):
        big[:, -tail:] = t[key]
    assert x.numel() > 2 ** 31
    y, last = M.moments_attn_fwd(M.attn_desc(x, k), x, k, q, da)
    a = [t[n] for n in ("xhat", "bhat", "qhat", "da")]
    y1, last1 = M.moments_attn_fwd(M.attn_desc(a[0], a[1]), *a)
    _check("y", y[:, -tail:], _np(y1), 2 * TOL[BF16])
    _check("h_last", last, _np(last1), 2 * TOL[F32])
    # and a slot of a pool of more than 2^31 values
    n = 2 ** 31 // (h * p * 16) + 2
    pool = torch.empty(n, h, p, 16, device=DEV)
    pool[n - 1] = last1[0]
    a = [v[:, -1:].contiguous() for v in a]
    d = M.attn_desc(a[0], a[1])
    own = last1.clone()
    y1 = M.moments_attn_step(d, *a, own)
    y = M.moments_attn_step(d, *a, pool, torch.tensor([n - 1], dtype=torch.int32, device=DEV))
    assert torch.equal(y, y1) and torch.equal(pool[n - 1], own[0])


def test_finite_check(monkeypatch):
    t = _make(1, 40, 1, 2, 2, 16, 16, F32, seed=16)
    a = [t[k] for k in ("xhat", "bhat", "qhat", "da", "h0")]
    d = M.attn_desc(a[0], a[1])
    monkeypatch.setenv("MOMENTS_CHECK_FINITE", "1")
    M.moments_attn_bwd(d, *a, t["d_y"], t["d_last"])
    a[0][0, 7, 0, 1, 3] = float("nan")
    with pytest.raises(M.MomentsError) as e:
        M.moments_attn_fwd(d, *a)
    assert e.value.code == M._lib.ENONFINITE
    with pytest.raises(M.MomentsError):
        M.moments_attn_bwd(d, *a, t["d_y"], t["d_last"])
