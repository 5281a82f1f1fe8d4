"""Edges of the gated recurrence, layer norm and the gradients' norm and clipping on the GPU."""
import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from bounds_util import same
from test_gpu_grad import both as clip_both, make as make_grads
from test_gpu_ln import both as ln_both, make as make_ln
from test_gpu_rec import make as make_rec, run_all
from test_gpu_recurrent import _example

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [M.GATE_LOG, M.GATE_MIX, M.GATE_UNIT])
@pytest.mark.parametrize("s", [60, 2200])
@pytest.mark.parametrize("clear,bad", [(18, 21), (18, 30), (50, 51), (8, 15)])
def test_a_cleared_state_keeps_later_nan_decays_out_of_earlier_gradients(dtype, gate, s, clear, bad):
    """A decay that is not a number behind a clearing one: in the same run of tokens, and in another."""
    t = make_rec(2, s, 12, gate, dtype, seed=s + clear)
    t["g"][:, clear] = -float("inf")
    clean = run_all(t, gate)
    t["g"][0, bad, 3] = float("nan")
    t["g"][1, bad, ::5] = float("nan")
    got = run_all(t, gate)
    for k in ("d_x", "d_g", "d_z"):      # what the clearing token hands to the left is zero
        assert same(got[k][:, :clear].contiguous(), clean[k][:, :clear].contiguous()), k
    assert same(got["d_h0"], clean["d_h0"])
    assert same(got["y"][:, :bad].contiguous(), clean["y"][:, :bad].contiguous())
    assert torch.isnan(got["y"][0, bad:, 3]).all() and torch.isnan(got["h_last"][0, 3])
    assert torch.isnan(got["d_x"][0, clear:bad, 3]).all()


def test_a_cleared_state_keeps_later_infinite_decays_out_of_earlier_gradients():
    """A clearing decay, two whose product underflows, an infinite one, all in one run of tokens."""
    t = make_rec(1, 60, 6, M.GATE_LOG, F32, z=False, seed=8)
    t["g"][:, 18] = -float("inf")
    clean = run_all(t, M.GATE_LOG)
    t["g"][0, 19:21, 2], t["g"][0, 21, 2] = -60.0, 95.0
    got = run_all(t, M.GATE_LOG)
    for k in ("d_x", "d_g"):
        assert same(got[k][:, :18].contiguous(), clean[k][:, :18].contiguous()), k
    assert same(got["d_h0"], clean["d_h0"])


@pytest.mark.parametrize("n", [3, 60])
def test_lengths_changed_before_the_backward_are_noticed(n):
    """A buffer of lengths that the next batch fills between a forward and its backward."""
    ex = _example()
    f = lambda *shape: torch.randn(*shape, device=DEV).requires_grad_()  # noqa: E731
    lens = torch.tensor([40, 7], dtype=torch.int32, device=DEV)
    y, _ = ex.Recurrence.apply(f(2, 80, 8), f(2, 80, 8), f(2, 80, 8), None, M.GATE_MIX, lens)
    lens.fill_(n)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_lengths_of_the_mixer_changed_before_the_backward_are_noticed():
    ex = _example("mixer")
    f = lambda *shape: torch.randn(*shape, device=DEV).requires_grad_()  # noqa: E731
    lens = torch.tensor([40, 7], dtype=torch.int32, device=DEV)
    y, _ = ex.Attention.apply(f(2, 80, 1, 2, 8), f(2, 80, 1, 2, 16), f(2, 80, 1, 2, 16), f(2, 80, 2), None, lens)
    lens.fill_(3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("w", [64, 33])
def test_the_last_tokens_of_long_projections(dtype, w):
    """One token of each sequence, more than 2^25 elements from the next one's: a step, a whole sequence
    of one token and its gradients, the same bits as of dense tokens."""
    wide = torch.zeros(3, 5, 7_000_000, dtype=dtype, device=DEV)
    assert wide.stride(0) > 2 ** 25
    t = make_rec(3, 1, w, M.GATE_UNIT, dtype, seed=w)
    far = {}
    for i, k in enumerate(("x", "g", "z")):
        far[k] = wide[:, -1:, i * w:(i + 1) * w]
        far[k].copy_(t[k])
    got, want = run_all({**t, **far}, M.GATE_UNIT), run_all(t, M.GATE_UNIT)
    for k in want:
        assert same(got[k], want[k]), k
    pool = torch.randn(5, w, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    ys, states = [], []
    for a in (far, t):
        states.append(pool.clone())
        d = M.rec_desc(a["x"], a["g"], a["z"], M.GATE_UNIT)
        ys.append(M.moments_rec_step(d, a["x"], a["g"], a["z"], states[-1], slots))
    assert same(*ys) and same(*states)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("w", [8200, 16384])
def test_several_wide_rows_to_a_workgroup(dtype, res, w):
    """Rows above 8192 columns, whose gradients' sums stand in LDS from row to row."""
    ln_both(make_ln(601, w, dtype, res=res, seed=w))


@pytest.mark.parametrize("n,w", [(40_003, 256), (140_001, 40)])
def test_more_narrow_rows_than_the_forward_takes_at_once(n, w):
    ln_both(make_ln(n, w, BF16, res=w == 40, seed=w))
    ln_both(make_ln(n, w, F32, res=w != 40, seed=w))


@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_more_pieces_than_workgroups(max_norm):
    """Gradients of more than 2048 pieces of 32 KB in a launch: later rounds of the workgroups, over tensors'
    borders, values outside 16-byte words among them."""
    sizes = [12_000_000, 4099, 9_000_001, 3, 5_000_003, 70_001]
    assert sum(n * 4 // 32768 for n in sizes[::2][:2]) > 2048
    clip_both(make_grads(sizes, dtypes=(F32, BF16), offset=3), max_norm)
    g = make_grads(sizes, dtypes=(F32, F32, F32, F32, BF16, BF16), seed=2, offset=1)
    clip_both(g, max_norm, out=[torch.empty(t.numel() + 2, dtype=t.dtype, device=DEV)[2:] for t in g])


def test_a_negative_norm_leaves_the_gradients():
    g = make_grads([100, 5000])
    copy = [t.clone() for t in g]
    M.moments_grad_clip(M.grad_desc(g), torch.full((), -2.0, device=DEV), 0.5)
    assert all(same(a, b) for a, b in zip(g, copy))
