"""Layer norm and its gradients on the GPU against the 64-bit oracle (oracle/layer_norm.py),
element by element within the bound that the oracle derives, plus one rounding of the output."""
import numpy as np
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from bounds_util import check, np64
from oracle import layer_norm

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def make(n, w, dtype, res=True, bias=True, stride=0, offset=0.0, start=0, seed=1):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    f = lambda *shape: torch.randn(*shape, device=DEV, generator=gen)  # noqa: E731
    x = (f(n, (stride or w) + start) + offset).to(dtype)[:, start:start + w]
    return {"x": x if stride or start else x.contiguous(), "res": 2 * f(n, w) if res else None,
            "weight": 1 + 0.3 * f(w), "bias": 0.5 * f(w) if bias else None, "d_y": f(n, w).to(dtype),
            "d_sum": f(n, w) if res else None}


def run(t, eps=EPS):
    d = M.ln_desc(t["x"], eps, t["res"] is not None)
    y, s = M.moments_ln_fwd(d, t["x"], t["weight"], t["bias"], t["res"])
    got = M.moments_ln_bwd(d, t["x"] if s is None else s, t["weight"], t["bias"], t["d_y"], t["d_sum"])
    got.update(y=y, sum=s)
    return got


def both(t, eps=EPS):
    n, w = t["x"].shape
    print(f"[case] {n} x {w} {t['x'].dtype} stride {t['x'].stride(0) if n else 0} res {t['res'] is not None}", flush=True)
    got = run(t, eps)
    a = {k: np64(v) for k, v in t.items()}
    # a workgroup's rows one after the other, then double
    o = layer_norm.ln(a["x"], a["res"], a["weight"], a["bias"], eps, a["d_y"], a["d_sum"], row_adds=min(n, 400))
    check("y", got["y"], o["y"], o["e_y"])
    check("d_x", got["d_x"], o["d_s"], o["e_d_s"])
    check("d_weight", got["d_weight"], o["d_weight"], o["e_d_weight"])
    if t["bias"] is not None:
        check("d_bias", got["d_bias"], o["d_bias"], o["e_d_bias"])
    if t["res"] is not None:
        check("sum", got["sum"], o["sum"], o["e_sum"])
        check("d_res", got["d_res"], o["d_s"], o["e_d_s"])
    else:
        assert got["sum"] is None and got["d_res"] is None
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("w", [1, 2, 7, 8, 64, 100, 511, 512, 520, 1000, 1024, 1025, 2040, 2048, 4095, 4096, 8184, 8192,
                               16383, 16384])
def test_widths(dtype, res, w):
    both(make(5, w, dtype, res=res, bias=w % 3 != 0, seed=w))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 2, 3, 33, 1000])
@pytest.mark.parametrize("w", [48, 129])
def test_rows(dtype, n, w):
    both(make(n, w, dtype, seed=n))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("w", [256, 1536])
def test_more_rows_than_places(dtype, w):
    """Several rows to each place of the launch, in the sums over rows too."""
    both(make(20_011, w, dtype, res=dtype is F32, seed=w))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("w,stride,start", [(64, 72, 0), (64, 65, 0), (64, 80, 8), (64, 80, 3), (33, 40, 1)])
def test_columns_of_a_wider_tensor(dtype, w, stride, start):
    for res in (True, False):
        both(make(9, w, dtype, res=res, stride=stride, start=start, seed=w + stride))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values_far_from_zero(dtype):
    both(make(50, 1000, dtype, res=False, offset=1000.0))
    if dtype is F32:
        both(make(50, 96, dtype, res=False, offset=1e6))


@pytest.mark.parametrize("w", [24, 129, 3000])
def test_rows_of_one_value(w):
    """No variance: y is the bias, and the gradients are those at rstd = 1 / sqrt(eps)."""
    for v in (0.0, 3.5, 1e30, 3e38):
        t = make(4, w, F32, res=False)
        t["x"][:] = v
        got = run(t)
        assert torch.equal(got["y"], t["bias"].expand(4, w))
        assert torch.count_nonzero(got["d_weight"]) == 0
        gy = np64(t["d_y"]) * np64(t["weight"])
        ref = (gy - gy.mean(-1, keepdims=True)) / np.sqrt(EPS)
        err = 70 * 2.0 ** -24 * (np.abs(gy) + np.abs(gy).mean(-1, keepdims=True)) / np.sqrt(EPS)
        check("d_x", got["d_x"], ref, err)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-25, 1e-15, 1e15, 1e22, 1e37])
def test_sizes_whose_squares_leave_the_range(dtype, scale):
    t = make(6, 300, dtype, res=False)
    t["x"] = (t["x"].float() * scale).to(dtype)
    both(t, 1e-30 if scale < 1 else EPS)


def test_rows_that_are_not_finite():
    t = make(9, 200, F32)
    clean = run(t)
    t["x"][2, 5], t["x"][4, 0], t["res"][6, 1] = float("nan"), float("inf"), -float("inf")
    got = run(t)
    ok = torch.ones(9, dtype=torch.bool, device=DEV)
    ok[[2, 4, 6]] = False
    for k in ("y", "d_x", "d_res"):
        assert torch.equal(got[k][ok], clean[k][ok]), k
        assert not torch.isfinite(got[k][~ok]).any()


def test_in_place_streams_and_wanted_only():
    for w in (96, 130):
        t = make(300, w, BF16)
        d = M.ln_desc(t["x"], EPS, True)
        ref = run(t)
        res, ds = t["res"].clone(), t["d_sum"].clone()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            y, s = M.moments_ln_fwd(d, t["x"], t["weight"], t["bias"], res, sum=res)
            g = M.moments_ln_bwd(d, s, t["weight"], t["bias"], t["d_y"], ds, out={"d_res": ds})
            assert s is res and g["d_res"] is ds
            for k in ("x", "res", "weight", "bias"):
                one = M.moments_ln_bwd(d, s, t["weight"], t["bias"], t["d_y"], t["d_sum"], want=(k,))
                assert torch.equal(one["d_" + k], ref["d_" + k])
                assert all(v is None for n, v in one.items() if n != "d_" + k)
            none = M.moments_ln_bwd(d, s, t["weight"], t["bias"], t["d_y"])       # no d_sum
        st.synchronize()
        assert torch.equal(y, ref["y"]) and torch.equal(res, ref["sum"])
        for k in ("d_x", "d_res", "d_weight", "d_bias"):
            assert torch.equal(g[k], ref[k]), k
        a = {k: np64(v) for k, v in t.items()}
        o = layer_norm.ln(a["x"], a["res"], a["weight"], a["bias"], EPS, a["d_y"])
        check("d_res", none["d_res"], o["d_s"], o["e_d_s"])


def test_no_rows():
    t = make(0, 40, F32)
    got = run(t)
    assert got["y"].shape == (0, 40) and got["d_res"].shape == (0, 40)
    assert torch.count_nonzero(got["d_weight"]) == 0 and torch.count_nonzero(got["d_bias"]) == 0


def test_leading_dimensions():
    x = torch.randn(3, 4, 5, 32, device=DEV)
    w = torch.ones(32, device=DEV)
    y, _ = M.moments_ln_fwd(M.ln_desc(x), x, w)
    y2, _ = M.moments_ln_fwd(M.ln_desc(x.view(60, 32)), x.view(60, 32), w)
    assert y.shape == x.shape and torch.equal(y.view(60, 32), y2)


def test_captured():
    t = make(70, 136, BF16)
    d = M.ln_desc(t["x"], EPS, True)

    def everything():
        y, s = M.moments_ln_fwd(d, t["x"], t["weight"], t["bias"], t["res"])
        g = M.moments_ln_bwd(d, s, t["weight"], t["bias"], t["d_y"], t["d_sum"])
        return [y, s, *(g[k] for k in sorted(g))]

    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = everything()
    for seed in (2, 3, 4):
        new = make(70, 136, BF16, seed=seed)
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, everything()):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    n, w = 70_000, 32_768
    wide = torch.zeros(n, w, dtype=BF16, device=DEV)
    assert wide.numel() > 2 ** 31
    t = make(3, 64, BF16, res=False)
    wide[-3:, :64] = t["x"]
    x = wide[:, :64]
    y, _ = M.moments_ln_fwd(M.ln_desc(x, EPS), x, t["weight"], t["bias"])
    o = layer_norm.ln(np64(t["x"]), None, np64(t["weight"]), np64(t["bias"]), EPS)
    check("y", y[-3:], o["y"], o["e_y"])


def test_finite_check(monkeypatch):
    monkeypatch.setenv("MOMENTS_CHECK_FINITE", "1")
    t = make(4, 16, F32)
    run(t)
    t["x"][1, 1] = float("nan")
    with pytest.raises(M.MomentsError) as e:
        run(t)
    assert e.value.code == M._lib.ENONFINITE
