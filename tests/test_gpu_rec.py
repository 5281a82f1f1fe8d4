"""The gated linear recurrence on the GPU against the 64-bit oracle (oracle/gated_rec.py),
element by element within the bound that the oracle derives for float32 arithmetic, plus
one rounding of the output."""
import numpy as np
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from bounds_util import check, np64, same
from oracle import gated_rec

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
GATES = (M.GATE_LOG, M.GATE_MIX, M.GATE_UNIT)


def make(b, s, w, gate, dtype, z=True, state=True, columns=False, lens=None, seed=1):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    f = lambda *shape: torch.randn(*shape, device=DEV, generator=gen)  # noqa: E731
    spread = torch.rand(w, device=DEV, generator=gen)
    g = f(b, s, w)
    g = -torch.nn.functional.softplus(g) * torch.exp(-8 * spread) if gate == M.GATE_LOG else g + 8 * spread - 1
    t = {"x": f(b, s, w).to(dtype), "g": g.to(dtype), "z": f(b, s, w).to(dtype) if z else None}
    if columns:   # cut out of a wider projection, `columns` values past its start
        names = [n for n in t if t[n] is not None]
        wide = torch.cat([f(b, s, columns).to(dtype)] + [t[n] for n in names] + [f(b, s, 5).to(dtype)], -1)
        t.update(zip(names, wide[:, :, columns:columns + len(names) * w].split(w, -1)))
    t["h0"] = f(b, w) if state else None
    t["d_y"] = f(b, s, w).to(dtype)
    t["d_h_last"] = f(b, w) if state else None
    t["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    return t


def desc(t, gate, valid_len=None):
    return M.rec_desc(t["x"], t["g"], t["z"], gate, valid_len=valid_len, valid_lens=t["lens"])


def run_all(t, gate, valid_len=None):
    """Forward, forward that saves and both backwards; the same bits where they compute the same."""
    d = desc(t, gate, valid_len)
    assert M.moments_rec_validate(d) == 0
    args = (t["x"], t["g"], t["z"], t["h0"])
    y, last = M.moments_rec_fwd(d, *args)
    y2, last2, saved = M.moments_rec_fwd_save(d, *args)
    got = M.moments_rec_bwd_saved(d, *args, saved, t["d_y"], t["d_h_last"])
    again = M.moments_rec_bwd(d, *args, t["d_y"], t["d_h_last"])
    assert same(y, y2) and same(last, last2)
    for k, v in got.items():
        assert (v is None) == (again[k] is None) and (v is None or same(v, again[k])), k
    got.update(y=y, h_last=last)
    return got


def compare(t, gate, got, valid_len=None):
    b, s, w = t["x"].shape
    top = s if valid_len is None else min(valid_len, s)
    lens = [top] * b if t["lens"] is None else [min(max(v, 0), top) for v in t["lens"].tolist()]
    n = {k: np64(v) for k, v in t.items()}
    o = gated_rec.rec(n["x"], n["g"], n["z"], n["h0"], gate, lens, n["d_y"], n["d_h_last"], bounds=True)
    for k in ("y", "h_last", "d_x", "d_g", "d_z", "d_h0"):
        if got[k] is None:
            assert (k == "d_z" and t["z"] is None) or (k == "d_h0" and t["h0"] is None)
            continue
        check(k, got[k], o[k], o["e_" + k])
    for i, v in enumerate(lens):
        for k in ("y", "d_x", "d_g", "d_z"):
            assert got[k] is None or torch.count_nonzero(got[k][i, v:]) == 0


def both(t, gate, valid_len=None):
    print(f"[case] gate {gate} {tuple(t['x'].shape)} {t['x'].dtype} stride {t['x'].stride()} z {t['z'] is not None}",
          flush=True)
    got = run_all(t, gate, valid_len)
    compare(t, gate, got, valid_len)
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("b,s,w", [(1, 1, 1), (2, 5, 2), (1, 64, 7), (3, 65, 128), (2, 129, 130), (1, 300, 257)])
def test_sizes(dtype, gate, b, s, w):
    both(make(b, s, w, gate, dtype, seed=s + w), gate)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("z,state", [(False, True), (True, False), (False, False)])
def test_without_output_gate_or_state(dtype, gate, z, state):
    both(make(2, 70, 34, gate, dtype, z=z, state=state), gate)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("s", [511, 2048, 4099])
def test_long_sequences_in_segments(dtype, gate, s):
    """Few channels: the sequence is split and its segments' states are joined."""
    both(make(1, s, 66, gate, dtype, seed=s), gate)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("w,columns", [(64, 8), (64, 2), (64, 1), (33, 3), (10, 64)])
def test_columns_of_a_projection(dtype, w, columns):
    for gate in GATES:
        both(make(2, 77, w, gate, dtype, columns=columns, seed=w), gate)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
def test_ragged_lengths(dtype, gate):
    t = make(6, 700, 40, gate, dtype, lens=[700, 0, 1, 513, -3, 10 ** 6])
    both(t, gate)
    both(t, gate, valid_len=300)
    both({**t, "lens": None}, gate, valid_len=0)
    both({**t, "lens": None}, gate, valid_len=650)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
def test_padding_may_hold_anything(dtype, gate):
    lens = [40, 0, 129]
    t = make(3, 200, 20, gate, dtype, lens=lens)
    clean = run_all(t, gate)
    for i, n in enumerate(lens):
        for k in ("x", "g", "z", "d_y"):
            t[k][i, n:] = float("nan")
    dirty = run_all(t, gate)
    for k in clean:
        assert torch.equal(clean[k], dirty[k]), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("s", [150, 2100])
def test_cleared_states(dtype, gate, s):
    """Decays of zero, at run, wave, tile and segment borders too."""
    t = make(2, s, 70, gate, dtype, seed=3)
    for at in (0, 7, 8, 63, 64, 100, 127, 128, s - 1):
        t["g"][0, at] = -float("inf")
        t["g"][1, at, ::3] = -200.0
    both(t, gate)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("s", [200, 2200])
def test_values_that_are_not_finite(dtype, gate, s):
    """They reach their channel's later tokens, up to a cleared state, and no other's; in the
    gradients, besides, its earlier ones."""
    t = make(2, s, 12, gate, dtype, seed=4)
    t["g"][:, 150] = -float("inf")
    clean = run_all(t, gate)
    t["x"][0, 20, 3] = float("inf")
    t["h0"][1, 5] = float("nan")
    t["h0"][1, 6] = float("inf")
    got = run_all(t, gate)
    bad = torch.zeros(2, s, 12, dtype=torch.bool, device=DEV)
    bad[0, 20:150, 3] = True
    bad[1, :150, 5] = True
    bad[1, :150, 6] = True
    assert not torch.isfinite(got["y"][bad].float()).any()
    assert torch.equal(got["y"][~bad], clean["y"][~bad])
    assert torch.equal(got["h_last"], clean["h_last"])
    grad = bad.clone()
    grad[0, :150, 3] = True
    for k in ("d_x", "d_g", "d_z"):
        assert torch.equal(got[k][~grad], clean[k][~grad]), k


def test_a_decay_that_only_underflows_keeps_what_is_not_finite():
    """A long product of decays underflows without clearing: an infinite state stays infinite."""
    for s in (100, 3000):
        t = make(1, s, 4, M.GATE_LOG, F32, z=False)
        t["g"][:] = -20.0
        t["h0"][0, 1] = float("inf")
        y, last = M.moments_rec_fwd(desc(t, M.GATE_LOG), t["x"], t["g"], None, t["h0"])
        assert not torch.isfinite(y[0, :, 1]).any() and not torch.isfinite(last[0, 1])
        assert torch.isfinite(y[0, :, [0, 2, 3]]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_extreme_gates(dtype):
    for gate in GATES:
        t = make(1, 90, 48, gate, dtype, seed=6)
        vals = [0.0, -0.0, -1e-7, -1e-3, -5.0, -80.0, -87.0, -88.0, -120.0]
        if gate != M.GATE_LOG:
            vals += [1e-3, 5.0, 20.0, 80.0, 100.0, float("inf")]
        for i, v in enumerate(vals):
            t["g"][0, :, 3 * i] = v
            t["g"][0, 40, 3 * i + 1] = v
        both(t, gate)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_growth(dtype):
    """Log-decays above zero: the state grows."""
    t = make(1, 130, 10, M.GATE_LOG, dtype)
    t["g"] = (t["g"].float() * 0.1 + 0.05).to(dtype)
    both(t, M.GATE_LOG)


@pytest.mark.parametrize("s", [120, 4000])
def test_growth_of_a_zero_state(s):
    """Log-decays above zero over tokens of zeros, whose product leaves the range, before the first value."""
    t = make(1, s, 6, M.GATE_LOG, F32, state=False)
    t["g"][:, :s - 40] = 1.0
    t["x"][:, :s - 40] = 0.0
    t["d_y"][:] = 0.0
    got = run_all(t, M.GATE_LOG)
    compare(t, M.GATE_LOG, got)
    assert torch.isfinite(got["y"]).all()


def test_last_state_may_be_the_first_and_pieces():
    """h_last in h0's buffer, d_h0 in d_h_last's, split into segments and not; a sequence in pieces."""
    for s in (60, 3000):
        t = make(2, s, 30, M.GATE_UNIT, F32, seed=9)
        d = desc(t, M.GATE_UNIT)
        y, last = M.moments_rec_fwd(d, t["x"], t["g"], t["z"], t["h0"])
        g = M.moments_rec_bwd(d, t["x"], t["g"], t["z"], t["h0"], t["d_y"], t["d_h_last"])
        h, dl = t["h0"].clone(), t["d_h_last"].clone()
        y2, same = M.moments_rec_fwd(d, t["x"], t["g"], t["z"], h, h_last=h)
        assert same is h and torch.equal(h, last) and torch.equal(y, y2)
        g2 = M.moments_rec_bwd(d, t["x"], t["g"], t["z"], t["h0"], t["d_y"], dl, out={"d_h0": dl})
        assert torch.equal(dl, g["d_h0"]) and torch.equal(g["d_g"], g2["d_g"])
        cut = s // 3
        parts, h = [], t["h0"]
        for sl in (slice(0, cut), slice(cut, s)):
            p = {k: t[k][:, sl].contiguous() for k in ("x", "g", "z")}
            y1, h = M.moments_rec_fwd(M.rec_desc(p["x"], p["g"], p["z"], M.GATE_UNIT), p["x"], p["g"], p["z"], h)
            parts.append(y1)
        compare(t, M.GATE_UNIT, {**g, "y": torch.cat(parts, 1), "h_last": h})


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("b,w,z", [(1, 1, True), (5, 37, False), (70, 130, True), (2, 600, True)])
def test_single_tokens(dtype, gate, b, w, z):
    """Steps against the oracle, slots scattered, unused rows and their slots left alone."""
    t = make(b, 3, w, gate, dtype, z=z, seed=b)
    pool = torch.randn(b + 4, w, device=DEV)
    slots = torch.randperm(b + 4, device=DEV)[:b].to(torch.int32)
    used = torch.ones(b, dtype=torch.bool)
    if b > 2:
        slots[1], slots[2] = -1, b + 4
        used[1] = used[2] = False
    state = pool.clone()
    ys = []
    for k in range(3):
        one = {n: None if t[n] is None else t[n][:, k:k + 1] for n in ("x", "g", "z")}
        d = M.rec_desc(one["x"], one["g"], one["z"], gate)
        ys.append(M.moments_rec_step(d, one["x"], one["g"], one["z"], state, slots))
    y = torch.cat(ys, 1)
    assert torch.count_nonzero(y[~used.to(DEV)]) == 0
    n = {k: np64(v) for k, v in t.items()}
    at = slots.long().cpu()[used]
    o = gated_rec.rec(*(None if n[k] is None else n[k][used.numpy()] for k in ("x", "g", "z")), np64(pool)[at.numpy()],
                      gate, bounds=True)
    check("y", y[used.to(DEV)], o["y"], o["e_y"])
    check("state", state[at.to(DEV)], o["h_last"], o["e_h_last"])
    rest = torch.ones(b + 4, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(state[rest.to(DEV)], pool[rest.to(DEV)])
    if b > 1:    # lengths of zero, and rows in order without slots
        state = pool.clone()
        one = {k: None if t[k] is None else t[k][:, :1] for k in ("x", "g", "z")}
        lens = torch.zeros(b, dtype=torch.int32, device=DEV)
        lens[0] = 1
        d = M.rec_desc(one["x"], one["g"], one["z"], gate, valid_lens=lens)
        y = M.moments_rec_step(d, one["x"], one["g"], one["z"], state)
        assert torch.count_nonzero(y[1:]) == 0 and torch.equal(state[1:], pool[1:])
        assert not torch.equal(state[0], pool[0])


def test_a_cleared_slot_forgets_what_is_not_finite():
    for gate in GATES:
        x = torch.ones(1, 1, 6, device=DEV)
        g = torch.full((1, 1, 6), -float("inf"), device=DEV)
        state = torch.full((1, 6), float("nan"), device=DEV)
        y = M.moments_rec_step(M.rec_desc(x, g, gate=gate), x, g, None, state)
        assert torch.equal(y, x) and torch.equal(state, x[0])


def test_nothing_to_do_and_wanted_only():
    t = make(2, 40, 12, M.GATE_MIX, BF16)
    d = desc(t, M.GATE_MIX)
    args = (t["x"], t["g"], t["z"], t["h0"])
    full = M.moments_rec_bwd(d, *args, t["d_y"], t["d_h_last"])
    for k in ("x", "g", "z", "h0"):
        one = M.moments_rec_bwd(d, *args, t["d_y"], t["d_h_last"], want=(k,))
        assert torch.equal(one["d_" + k], full["d_" + k])
        assert all(v is None for n, v in one.items() if n != "d_" + k)
    e = {k: t[k][:, :0] for k in ("x", "g", "z", "d_y")}
    d = M.rec_desc(e["x"], e["g"], e["z"], M.GATE_MIX)
    y, last = M.moments_rec_fwd(d, e["x"], e["g"], e["z"], t["h0"])
    assert y.shape == (2, 0, 12) and torch.equal(last, t["h0"])
    g = M.moments_rec_bwd(d, e["x"], e["g"], e["z"], t["h0"], e["d_y"], t["d_h_last"])
    assert g["d_x"].shape == (2, 0, 12) and torch.equal(g["d_h0"], t["d_h_last"])
    _, last = M.moments_rec_fwd(d, e["x"], e["g"], e["z"])
    assert torch.count_nonzero(last) == 0
    n = {k: t[k][:0] for k in ("x", "g", "z", "h0", "d_y", "d_h_last")}
    d = M.rec_desc(n["x"], n["g"], n["z"], M.GATE_MIX)
    y, last = M.moments_rec_fwd(d, n["x"], n["g"], n["z"], n["h0"])
    assert y.shape == (0, 40, 12) and last.shape == (0, 12)
    assert M.moments_rec_bwd(d, n["x"], n["g"], n["z"], n["h0"], n["d_y"])["d_x"].shape == (0, 40, 12)


def test_gradient_against_differences():
    rng = np.random.default_rng(2)
    for gate in GATES:
        t = make(1, 30, 9, gate, F32, seed=13)
        got = run_all(t, gate)
        n = {k: np64(v) for k, v in t.items()}

        def loss(a):
            o = gated_rec.rec(a["x"], a["g"], a["z"], a["h0"], gate)
            return (o["y"] * n["d_y"]).sum() + (o["h_last"] * n["d_h_last"]).sum()

        for k in ("x", "g", "z", "h0"):
            v = rng.standard_normal(n[k].shape)
            num = (loss({**n, k: n[k] + 1e-6 * v}) - loss({**n, k: n[k] - 1e-6 * v})) / 2e-6
            g = np64(got["d_" + k])
            # 30 tokens of a few roundings each in float32, and the differences' own error
            assert abs((g * v).sum() - num) <= 1e-5 * np.linalg.norm(g) * np.linalg.norm(v) + 1e-7 * abs(num), k


def test_streams_and_repetition():
    """The same bits on another stream, twice, and with calls of other sizes between."""
    t = make(2, 1500, 50, M.GATE_UNIT, BF16, seed=17)
    first = run_all(t, M.GATE_UNIT)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run_all(make(1, 300, 40, M.GATE_LOG, F32), M.GATE_LOG)
        second = run_all(t, M.GATE_UNIT)
    st.synchronize()
    for k in first:
        assert torch.equal(first[k], second[k]), k


@pytest.mark.parametrize("s,w", [(90, 40), (2500, 70)])
def test_captured(s, w):
    """Forward, backward and a step in one graph, replayed on new inputs."""
    t = make(2, s, w, M.GATE_MIX, BF16, seed=21)
    d = desc(t, M.GATE_MIX)
    args = (t["x"], t["g"], t["z"], t["h0"])
    one = tuple(v[:, :1].contiguous() for v in args[:3])
    d1 = M.rec_desc(*one, M.GATE_MIX)
    state = torch.zeros(2, w, device=DEV)

    def everything():
        y, last, saved = M.moments_rec_fwd_save(d, *args)
        g = M.moments_rec_bwd_saved(d, *args, saved, t["d_y"], t["d_h_last"])
        return [y, last, M.moments_rec_step(d1, *one, state), *(g[k] for k in sorted(g))]

    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = everything()
    for seed in (1, 2, 3):
        new = make(2, s, w, M.GATE_MIX, BF16, seed=seed)
        for k in ("x", "g", "z", "h0", "d_y", "d_h_last"):
            t[k].copy_(new[k])
        state.fill_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        state.fill_(0.5)
        for a, b in zip(got, everything()):
            assert torch.equal(a, b)


def test_more_chains_than_the_card_holds_at_once():
    """Several rounds of workgroups, and a count of them that is no multiple of the card's."""
    for b, s, w, dtype in ((300, 40, 130, BF16), (37, 260, 1100, F32)):
        both(make(b, s, w, M.GATE_MIX, dtype, seed=b), M.GATE_MIX)


def test_two_calls_at_once():
    """Two streams, each with its own workspace, in segments."""
    t = [make(2, 2100, 70, M.GATE_UNIT, BF16, seed=k) for k in (1, 2)]
    want = [run_all(v, M.GATE_UNIT) for v in t]
    streams = [torch.cuda.Stream() for _ in t]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for v, st in zip(t, streams):
            with torch.cuda.stream(st):
                d = desc(v, M.GATE_UNIT)
                y, last, saved = M.moments_rec_fwd_save(d, v["x"], v["g"], v["z"], v["h0"])
                g = M.moments_rec_bwd_saved(d, v["x"], v["g"], v["z"], v["h0"], saved, v["d_y"], v["d_h_last"])
                got.append({**g, "y": y, "h_last": last})
        for st in streams:
            st.synchronize()
        for a, b in zip(want, got):
            for k in a:
                assert torch.equal(a[k], b[k]), k


def test_offsets_past_32_bits():
    """Rows cut out of a projection of more than 2^31 values."""
    s, width = 70_000, 32_768
    wide = torch.zeros(1, s, width, dtype=BF16, device=DEV)
    assert wide.numel() > 2 ** 31
    t = make(1, 6, 8, M.GATE_MIX, BF16, seed=5)
    for i, k in enumerate(("x", "g", "z")):
        wide[:, -6:, 8 * i:8 * i + 8] = t[k]
    x, g, z = wide[:, :, :8], wide[:, :, 8:16], wide[:, :, 16:24]
    y, last = M.moments_rec_fwd(M.rec_desc(x, g, z, M.GATE_MIX), x, g, z)   # zeros leave the state at zero
    ref = gated_rec.rec(np64(t["x"]), np64(t["g"]), np64(t["z"]), None, M.GATE_MIX, bounds=True)
    check("y", y[:, -6:], ref["y"], ref["e_y"])
    check("h_last", last, ref["h_last"], ref["e_h_last"])


def test_finite_check(monkeypatch):
    monkeypatch.setenv("MOMENTS_CHECK_FINITE", "1")
    t = make(1, 20, 6, M.GATE_LOG, F32)
    run_all(t, M.GATE_LOG)
    t["x"][0, 3, 2] = float("nan")
    with pytest.raises(M.MomentsError) as e:
        M.moments_rec_fwd(desc(t, M.GATE_LOG), t["x"], t["g"], t["z"], t["h0"])
    assert e.value.code == M._lib.ENONFINITE
