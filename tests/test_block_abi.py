"""Refusals of the gated recurrence, layer norm and the gradients' norm and clipping, on the
host: bad descriptors, missing or misaligned pointers, small buffers, and the Python binding's
checks. No GPU is touched."""
import ctypes

import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from mamba_ssm_chunkwise_amd import _lib

FAKE, NULL = ctypes.c_void_p(1 << 20), ctypes.c_void_p()
ODD, BYTE = ctypes.c_void_p((1 << 20) + 4), ctypes.c_void_p((1 << 20) + 1)
BIG = 1 << 50
F32, BF16 = torch.float32, torch.bfloat16


def _rec(**kw):
    d = dict(b=2, s=64, w=10, valid_len=64, x_stride=0, g_stride=0, z_stride=0, dtype=_lib.F32, gate=0, has_z=1,
             reserved=0)
    d.update(kw)
    return M.RecDesc(**d)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(dtype=_lib.BF16, gate=2), 0), (dict(gate=1, has_z=0), 0), (dict(s=0), 0), (dict(b=0), 0),
    (dict(valid_len=0), 0), (dict(valid_len=10 ** 12), 0), (dict(w=1), 0), (dict(w=1 << 24, b=1), 0),
    (dict(x_stride=10, g_stride=11, z_stride=40), 0), (dict(has_z=0, z_stride=3), 0),
    (dict(w=0), -1), (dict(s=-1), -1), (dict(b=-1), -1), (dict(valid_len=-1), -1), (dict(dtype=2), -1),
    (dict(gate=3), -1), (dict(gate=-1), -1), (dict(has_z=2), -1), (dict(reserved=1), -1), (dict(x_stride=9), -1),
    (dict(g_stride=-1), -1), (dict(z_stride=9), -1),
    (dict(w=(1 << 24) + 1), -2), (dict(s=2 ** 29), -2), (dict(b=2 ** 25), -2), (dict(x_stride=1 << 41), -2),
    (dict(b=2 ** 23, w=64), -2), (dict(b=1 << 10, w=1 << 20), -2),
])
def test_rec_descriptor(kw, code):
    lib, d = _lib.load(), _rec(**kw)
    assert M.moments_rec_validate(d) == code
    for n in (lib.moments_rec_workspace_size(ctypes.byref(d), 0), lib.moments_rec_workspace_size(ctypes.byref(d), 1),
              lib.moments_rec_saved_size(ctypes.byref(d))):
        assert (n >= 0) if code == 0 else (n == code)


def test_null_descriptors():
    lib = _lib.load()
    assert lib.moments_rec_validate(None) == -1 and lib.moments_rec_saved_size(None) == -1
    assert lib.moments_ln_workspace_size(None) == -1
    assert lib.moments_rec_fwd(None, *[FAKE] * 6, FAKE, BIG, NULL) == -1
    assert lib.moments_ln_fwd(None, *[FAKE] * 6, NULL) == -1
    assert lib.moments_ln_bwd(None, *[FAKE] * 8, FAKE, BIG, NULL) == -1
    assert lib.moments_grad_validate(None, 1) == -1 and lib.moments_grad_workspace_size(None, 1) == -1
    assert lib.moments_grad_validate(None, 0) == 0


def test_rec_pointers_and_buffers():
    lib, d = _lib.load(), ctypes.byref(_rec(s=3000, valid_len=3000))
    ok = [FAKE] * 6                                        # x g z h0 y h_last
    fwd = lambda *a: lib.moments_rec_fwd(d, *a)            # noqa: E731
    for i in range(6):
        bad = list(ok)
        if i not in (3, 5):
            bad[i] = NULL
            assert fwd(*bad, FAKE, BIG, NULL) == -1
        bad[i] = BYTE if i < 3 else ODD                    # x, g and z may start at any element
        assert fwd(*bad, FAKE, BIG, NULL) == -1
    assert fwd(*ok, NULL, BIG, NULL) == -3
    assert fwd(*ok, FAKE, 16, NULL) == -3
    assert fwd(*ok, ODD, BIG, NULL) == -1
    assert lib.moments_rec_fwd_save(d, *ok, NULL, BIG, FAKE, BIG, NULL) == -1
    assert lib.moments_rec_fwd_save(d, *ok, FAKE, 16, FAKE, BIG, NULL) == -3
    args = [FAKE] * 10                                     # x g z h0 d_y d_h_last d_x d_g d_z d_h0
    for i in (0, 1, 2, 4):
        bad = list(args)
        bad[i] = NULL
        assert lib.moments_rec_bwd(d, *bad, FAKE, BIG, NULL) == -1
    for i in range(3, 10):
        bad = list(args)
        bad[i] = ODD
        assert lib.moments_rec_bwd(d, *bad, FAKE, BIG, NULL) == -1
    assert lib.moments_rec_bwd(d, *args, FAKE, 16, NULL) == -3
    assert lib.moments_rec_bwd_saved(d, *args[:4], FAKE, 16, *args[4:], FAKE, BIG, NULL) == -3
    assert lib.moments_rec_bwd_saved(d, *args[:4], NULL, BIG, *args[4:], FAKE, BIG, NULL) == -1
    none = ctypes.byref(_rec(has_z=0))
    assert lib.moments_rec_fwd(none, *ok, FAKE, BIG, NULL) == -1                       # z without has_z
    assert lib.moments_rec_bwd(none, FAKE, FAKE, NULL, *args[3:], FAKE, BIG, NULL) == -1   # d_z


def test_rec_step_refusals():
    lib, one = _lib.load(), _rec(s=1)
    step = lambda d, *a: lib.moments_rec_step(ctypes.byref(d), *a)   # noqa: E731
    assert step(_rec(s=2), FAKE, FAKE, FAKE, NULL, 9, FAKE, FAKE, NULL) == -1
    assert step(one, FAKE, FAKE, FAKE, NULL, 1, FAKE, FAKE, NULL) == -1       # fewer slots than rows
    assert step(one, FAKE, FAKE, FAKE, FAKE, -1, FAKE, FAKE, NULL) == -1
    assert step(one, FAKE, FAKE, FAKE, FAKE, (1 << 30) + 1, FAKE, FAKE, NULL) == -1
    assert step(one, FAKE, FAKE, FAKE, FAKE, 4, NULL, FAKE, NULL) == -1
    assert step(one, FAKE, FAKE, NULL, FAKE, 4, FAKE, FAKE, NULL) == -1
    assert step(one, FAKE, FAKE, FAKE, BYTE, 4, FAKE, FAKE, NULL) == -1
    assert step(one, FAKE, FAKE, FAKE, FAKE, 4, FAKE, ODD, NULL) == -1


def _ln(**kw):
    d = dict(n=5, w=16, x_stride=0, dtype=_lib.F32, residual=1, eps=1e-5, reserved=0)
    d.update(kw)
    return M.LnDesc(**d)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(n=0), 0), (dict(w=1), 0), (dict(w=16384), 0), (dict(x_stride=17), 0), (dict(eps=1e-30), 0),
    (dict(residual=0, dtype=_lib.BF16), 0),
    (dict(n=-1), -1), (dict(w=0), -1), (dict(x_stride=15), -1), (dict(dtype=5), -1), (dict(residual=2), -1),
    (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(reserved=1), -1), (dict(w=16385), -2), (dict(n=1 << 41), -2), (dict(x_stride=1 << 41), -2),
])
def test_ln_descriptor(kw, code):
    n = _lib.load().moments_ln_workspace_size(ctypes.byref(_ln(**kw)))
    assert (n >= 0) if code == 0 else (n == code)


def test_ln_pointers_and_buffers():
    lib = _lib.load()
    d, plain = ctypes.byref(_ln()), ctypes.byref(_ln(residual=0))
    ok = [FAKE] * 6                                        # x res weight bias y sum
    for i in (0, 1, 2, 4, 5):
        bad = list(ok)
        bad[i] = NULL
        assert lib.moments_ln_fwd(d, *bad, NULL) == -1
    for i in range(6):
        bad = list(ok)
        bad[i] = BYTE if i == 0 else ODD
        assert lib.moments_ln_fwd(d, *bad, NULL) == -1
    assert lib.moments_ln_fwd(plain, *ok, NULL) == -1                           # res without a residual
    args = [FAKE] * 8                                      # x weight d_y d_sum d_x d_res d_weight d_bias
    for i in (0, 1, 2):
        bad = list(args)
        bad[i] = NULL
        assert lib.moments_ln_bwd(d, *bad, FAKE, BIG, NULL) == -1
    for i in range(1, 8):
        bad = list(args)
        bad[i] = ODD
        assert lib.moments_ln_bwd(d, *bad, FAKE, BIG, NULL) == -1
    assert lib.moments_ln_bwd(d, *args, FAKE, 16, NULL) == -3
    assert lib.moments_ln_bwd(d, *args, NULL, BIG, NULL) == -3
    assert lib.moments_ln_bwd(plain, *args, FAKE, BIG, NULL) == -1              # d_sum without a residual


def _spans(*rows):
    return (_lib.Span * len(rows))(*[_lib.Span(*r) for r in rows])


def test_grad_refusals():
    lib, A = _lib.load(), 1 << 20
    ok = _spans((A, None, 100, 0, 0), (A + 400, A + 800, 100, 0, 0))
    assert lib.moments_grad_validate(ok, 2) == 0
    for bad in ((0, None, 1, 0, 0), (A + 2, None, 1, 0, 0), (A + 1, None, 1, 1, 0), (A, A + 3, 1, 0, 0),
                (A, None, -1, 0, 0), (A, None, 1, 2, 0), (A, None, 1, 0, 7)):
        assert lib.moments_grad_validate(_spans(bad), 1) == -1
        assert lib.moments_grad_workspace_size(_spans(bad), 1) == -1
        assert lib.moments_grad_norm(_spans(bad), 1, FAKE, FAKE, BIG, NULL) == -1
        assert lib.moments_grad_clip(_spans(bad), 1, FAKE, 1.0, NULL) == -1
    assert lib.moments_grad_validate(_spans((A, None, 1 << 41, 0, 0)), 1) == -2
    assert lib.moments_grad_validate(ok, -1) == -1 and lib.moments_grad_validate(ok, 1 << 21) == -2
    assert lib.moments_grad_validate(_spans((0, None, 0, 0, 0)), 1) == 0        # empty: nothing is read
    assert lib.moments_grad_norm(ok, 2, NULL, FAKE, BIG, NULL) == -1
    assert lib.moments_grad_norm(ok, 2, FAKE, FAKE, 8, NULL) == -3
    assert lib.moments_grad_norm(ok, 2, FAKE, NULL, BIG, NULL) == -3
    for bad in (-1.0, float("nan")):
        assert lib.moments_grad_clip(ok, 2, FAKE, bad, NULL) == -1
    assert lib.moments_grad_clip(ok, 2, NULL, 1.0, NULL) == -1


@pytest.mark.parametrize("rows,code", [
    ([(0, None, 10), (40, None, 10)], 0),                  # neighbours
    ([(0, None, 10), (36, None, 10)], -1),                 # one value shared, both written
    ([(0, None, 10), (0, None, 10)], -1),                  # listed twice
    ([(0, 100, 10), (0, 200, 10)], 0),                     # read twice, written apart
    ([(0, 100, 10), (60, 120, 10)], -1),                   # outputs overlap
    ([(0, 40, 10), (40, 400, 10)], -1),                    # one's output is another's input
    ([(0, 20, 10)], -1),                                   # an output that overlaps its own input
    ([(0, 0, 10)], 0),                                     # in place, named
    ([(0, 400, 100), (40, 1000, 2), (80, None, 2)], -1),   # inside a longer one
    ([(0, None, 0), (0, None, 10)], 0),
])
def test_grad_overlaps(rows, code):
    A = 1 << 20
    s = _spans(*[(A + p, None if o is None else A + o, n, 0, 0) for p, o, n in rows])
    assert _lib.load().moments_grad_validate(s, len(rows)) == code


def test_binding_checks():
    x = torch.zeros(2, 6, 8)
    for bad in (lambda: M.rec_desc(x[0], x, gate=0), lambda: M.rec_desc(x, x.transpose(1, 2), gate=0),
                lambda: M.rec_desc(x.expand(2, 6, 8)[:, :, ::2], x[:, :, ::2]), lambda: M.rec_desc("x", x),
                lambda: M.rec_desc(x, x, valid_lens=torch.zeros(2, dtype=torch.int32)),
                lambda: M.ln_desc(torch.zeros(())), lambda: M.ln_desc(x.transpose(0, 1)),
                lambda: M.ln_desc(x[:, :, ::2]), lambda: M.grad_desc([x, torch.zeros(3, dtype=torch.float16)]),
                lambda: M.grad_desc([x.transpose(0, 1)]), lambda: M.grad_desc([x, x]), lambda: M.grad_desc([x[0], x]),
                lambda: M.grad_desc([x], out=[]), lambda: M.grad_desc([x], out=[x.bfloat16()]),
                lambda: M.grad_desc([x], out=[x[:1]]), lambda: M.grad_desc([None])):
        with pytest.raises(ValueError):
            bad()
    d = M.rec_desc(x, x, x)
    h0 = torch.zeros(2, 8)
    for bad in (lambda: M.moments_rec_fwd(d, x, x),                                # z missing
                lambda: M.moments_rec_fwd(M.rec_desc(x, x), x, x, x),              # z too many
                lambda: M.moments_rec_fwd(d, x, x, x[:, :5]), lambda: M.moments_rec_fwd(d, x, x.bfloat16(), x),
                lambda: M.moments_rec_fwd(d, x, torch.zeros(2, 6, 16)[:, :, :8], x),   # another stride
                lambda: M.moments_rec_fwd(d, x, x, x, h0.double()), lambda: M.moments_rec_fwd(d, x, x, x, h0[:1]),
                lambda: M.moments_rec_fwd(d, x, x, x, y=x[:1]), lambda: M.moments_rec_bwd(d, x, x, x, None, x[:1]),
                lambda: M.moments_rec_bwd_saved(d, x, x, x, None, None, x),
                lambda: M.moments_rec_step(d, x, x, x, h0[None]),
                lambda: M.moments_rec_fwd(d, x, x, x)):                            # no GPU tensors
        with pytest.raises(ValueError):
            bad()
    w = torch.ones(8)
    d, r = M.ln_desc(x), M.ln_desc(x, residual=True)
    for bad in (lambda: M.moments_ln_fwd(d, x, None), lambda: M.moments_ln_fwd(d, x, w[:4]),
                lambda: M.moments_ln_fwd(d, x, w, res=x), lambda: M.moments_ln_fwd(r, x, w),
                lambda: M.moments_ln_fwd(r, x, w, res=x.bfloat16()), lambda: M.moments_ln_fwd(d, x.bfloat16(), w),
                lambda: M.moments_ln_fwd(d, x[:1], w), lambda: M.moments_ln_bwd(d, x, w, None, x, x),
                lambda: M.moments_ln_bwd(r, x.bfloat16(), w, None, x),
                lambda: M.moments_ln_fwd(d, x, w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        M.moments_grad_norm(M.grad_desc([x]))
    with pytest.raises(ValueError):
        M.moments_grad_norm(M.grad_desc([]))
    with pytest.raises(M.MomentsError):
        M._size(_lib.load().moments_ln_workspace_size(ctypes.byref(M.ln_desc(x, eps=0.0))))


def test_gradients_that_moved():
    """A descriptor holds addresses: tensors that got other memory since are refused."""
    for move in (lambda t: t.resize_(4096), lambda t: t.untyped_storage().resize_(0),
                 lambda t: setattr(t, "data", torch.zeros(40))):
        for moved in (0, 1):
            g, o = torch.zeros(40), torch.zeros(40)
            d = M.grad_desc([g], out=[o])
            move((g, o)[moved])
            for call in (lambda: M.moments_grad_norm(d), lambda: M.moments_grad_clip(d, torch.zeros(()), 1.0)):
                with pytest.raises(ValueError, match="other memory"):
                    call()
