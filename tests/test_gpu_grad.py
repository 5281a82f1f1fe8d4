"""The gradients' norm and clipping on the GPU against 64 bits. The norm: sums in double, one
rounding of the result and that of the root: 2^-23. The clipped values: the factor is a
quotient of two float32 numbers that may each be off by three roundings, one more for the
product, then one rounding of the output."""
import math

import numpy as np
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from bounds_util import check, np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def make(sizes, dtypes=(F32, BF16), scale=1.0, seed=1, offset=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        v = torch.randn(n + offset, device=DEV, generator=gen) * scale
        out.append(v.to(dtypes[i % len(dtypes)])[offset:])
    return out


def exact(grads):
    return math.sqrt(sum(float((np64(g) ** 2).sum()) for g in grads))


def both(grads, max_norm, out=None):
    before = [np64(g) for g in grads]
    want = exact(grads)
    d = M.grad_desc(grads, out=out)
    norm = M.moments_grad_norm(d)
    assert norm.dtype is F32 and norm.shape == ()
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    res = M.moments_grad_clip(d, norm, max_norm)
    f = min(1.0, max_norm / (want + 1e-6))
    for i, (r, b) in enumerate(zip(res, before)):
        ref = b * f
        # a norm within 2^-22 of the limit may fall on either side of it: the factor is 1 to 2^-22
        check(f"{i}", r, ref, 2.0 ** -21 * np.abs(ref))
    if out is not None:
        for g, b in zip(grads, before):
            assert np.array_equal(np64(g), b)
    return norm, res


@pytest.mark.parametrize("sizes", [[1], [3, 5], [0, 7, 0], [32768], [32769, 1], [8193, 16384, 1, 70_001], [1 << 22, 9]])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_sizes(sizes, max_norm):
    both(make(sizes), max_norm)
    g = make(sizes, dtypes=(BF16, F32), seed=2)
    both(g, max_norm, out=[torch.empty_like(t) for t in g])


@pytest.mark.parametrize("count", [63, 64, 65, 300])
def test_many_tensors(count):
    """More tensors than one launch takes, empty ones among them."""
    both(make([(37 * i) % 5000 for i in range(count)]), 1.0)


@pytest.mark.parametrize("offset", [1, 3, 5])
def test_tensors_that_start_anywhere(offset):
    sizes = [1, 2, 6, 7, 8, 9, 40_003]
    both(make(sizes, offset=offset), 0.1)
    g = make(sizes, offset=offset)
    both(g, 0.1, out=[torch.empty(t.numel() + 2, dtype=t.dtype, device=DEV)[2:] for t in g])


def test_neighbours_are_left_alone():
    for dtype in (F32, BF16):
        whole = torch.ones(1000, dtype=dtype, device=DEV)
        both([whole[3:500], whole[501:994]], 0.25)
        assert float(whole[:3].float().sum()) == 3 and whole[500] == 1 and float(whole[994:].float().sum()) == 6


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e19, 1e30])
def test_squares_out_of_range(scale):
    both(make([1000, 300], scale=scale), 1.0)


def test_limits():
    g = make([100, 200])
    want = exact(g)
    copy = [t.clone() for t in g]
    norm, _ = both(g, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(g, copy))
    M.moments_grad_clip(M.grad_desc(g), norm, want * 2)          # below the limit: the same bits
    assert all(torch.equal(a, b) for a, b in zip(g, copy))
    M.moments_grad_clip(M.grad_desc(g), norm, 0.0)
    assert all(torch.count_nonzero(t) == 0 for t in g)
    norm, _ = both(g, 1.0)
    assert float(norm) == 0.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    g = make([100, 5000])
    g[1][4321] = bad
    copy = [t.clone() for t in g]
    out = [torch.zeros_like(t) for t in g]
    d = M.grad_desc(g, out=out)
    norm = M.moments_grad_norm(d)
    assert not torch.isfinite(norm)
    M.moments_grad_clip(d, norm, 1.0)
    M.moments_grad_clip(M.grad_desc(g), norm, 1.0)
    for a, b, c in zip(g, copy, out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(c.view(torch.uint8), b.view(torch.uint8))


def test_no_gradients():
    d = M.grad_desc([])
    norm = torch.full((), 3.0, device=DEV)
    assert M.moments_grad_norm(d, norm=norm) is norm and float(norm) == 0.0
    assert M.moments_grad_clip(d, norm, 1.0) == []
    d = M.grad_desc([torch.empty(0, device=DEV)])
    assert float(M.moments_grad_norm(d)) == 0.0


def test_a_norm_over_ranks():
    """Shares' norms joined on the device, then both clipped by the joint one."""
    a, b = make([500, 70]), make([900], seed=3)
    want = exact(a + b)
    da, db = M.grad_desc(a), M.grad_desc(b)
    joint = torch.hypot(M.moments_grad_norm(da), M.moments_grad_norm(db))
    ref = [np64(t) * (1.0 / (want + 1e-6)) for t in a + b]
    for r, t in zip(ref, M.moments_grad_clip(da, joint, 1.0) + M.moments_grad_clip(db, joint, 1.0)):
        check("joint", t, r, 2.0 ** -20 * np.abs(r))


def test_shapes_streams_and_repetition():
    g = [torch.randn(3, 4, 5, device=DEV), torch.randn((), device=DEV), torch.randn(700, 900, device=DEV).bfloat16()]
    d = M.grad_desc(g)
    first = M.moments_grad_norm(d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(3):
            assert torch.equal(M.moments_grad_norm(d), first)
        M.moments_grad_clip(d, first, 1.0)
    st.synchronize()
    assert abs(exact(g) - 1.0) < 2.0 ** -7      # bf16 values, each within a rounding of 2^-8


def test_captured():
    g = make([1000, 40_000, 3])
    out = [torch.empty_like(t) for t in g]
    d = M.grad_desc(g, out=out)

    def everything():
        norm = M.moments_grad_norm(d)
        M.moments_grad_clip(d, norm, 1.0)
        return norm

    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = everything()
    for seed in (2, 3, 4):
        for t, v in zip(g, make([1000, 40_000, 3], seed=seed, scale=seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [norm.clone()] + [o.clone() for o in out]
        for a, b in zip(got, [everything(), *out]):
            assert torch.equal(a, b)


def test_finite_check(monkeypatch):
    monkeypatch.setenv("MOMENTS_CHECK_FINITE", "1")
    g = make([10])
    M.moments_grad_norm(M.grad_desc(g))
    g[0][3] = float("nan")
    with pytest.raises(M.MomentsError) as e:
        M.moments_grad_norm(M.grad_desc(g))
    assert e.value.code == M._lib.ENONFINITE
