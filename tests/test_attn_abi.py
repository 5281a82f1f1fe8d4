"""Refusals of the linear attention and of the norms with rotation, on the host:
bad descriptors, missing or misaligned pointers, small buffers, and the Python
binding's checks of shapes, types, strides and devices. No GPU is touched."""
import ctypes

import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from mamba_ssm_chunkwise_amd import _lib

FAKE, NULL, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p(), ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 50


def _attn(**kw):
    d = dict(b=2, s=64, c=2, h=4, g=2, p=8, r=16, valid_len=64, dtype=M._lib.F32, reserved=0)
    d.update(kw)
    return M.AttnDesc(**d)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(dtype=_lib.BF16), 0), (dict(s=61), 0), (dict(s=0), 0), (dict(b=0), 0), (dict(h=0), 0),
    (dict(valid_len=0), 0), (dict(valid_len=10 ** 9), 0), (dict(p=4096), 0), (dict(r=128), 0), (dict(r=1, p=1), 0),
    (dict(g=3), -1), (dict(g=0), -1), (dict(c=0), -1), (dict(p=0), -1), (dict(r=0), -1), (dict(s=-1), -1),
    (dict(valid_len=-1), -1), (dict(dtype=4), -1),
    (dict(r=129), -2), (dict(c=5), -2), (dict(p=4097), -2), (dict(s=2 ** 29), -2), (dict(b=2 ** 30), -2),
])
def test_attn_descriptor(kw, code):
    lib, d = _lib.load(), _attn(**kw)
    assert M.moments_attn_validate(d) == code
    for n in (lib.moments_attn_workspace_size(ctypes.byref(d), 1), lib.moments_attn_saved_size(ctypes.byref(d))):
        assert (n >= 0) if code == 0 else (n == code)


def test_attn_null_descriptor():
    lib = _lib.load()
    assert lib.moments_attn_validate(None) == -1
    assert lib.moments_qk_workspace_size(None) == -1


def test_attn_pointers_and_buffers():
    lib, d = _lib.load(), ctypes.byref(_attn())
    fwd = lambda *a: lib.moments_attn_fwd(d, *a)  # noqa: E731
    ok = [FAKE] * 4 + [NULL, FAKE, NULL]
    for i in (0, 1, 2, 3, 5):
        bad = list(ok)
        bad[i] = NULL
        assert fwd(*bad, FAKE, BIG, NULL) == -1
        bad[i] = ODD
        assert fwd(*bad, FAKE, BIG, NULL) == -1
    assert fwd(*ok, NULL, BIG, NULL) == -3
    assert fwd(*ok, FAKE, 16, NULL) == -3
    assert lib.moments_attn_fwd_save(d, *ok, NULL, BIG, FAKE, BIG, NULL) == -1
    assert lib.moments_attn_fwd_save(d, *ok, FAKE, 16, FAKE, BIG, NULL) == -3
    args = [FAKE] * 4 + [NULL, NULL, NULL] + [FAKE] * 5
    assert lib.moments_attn_bwd(d, *args, FAKE, BIG, NULL) == -1           # no d_y
    args[5] = FAKE
    assert lib.moments_attn_bwd(d, *args, FAKE, 16, NULL) == -3
    args[8] = ODD
    assert lib.moments_attn_bwd(d, *args, FAKE, BIG, NULL) == -1
    # nothing to do: nothing is looked at
    assert lib.moments_attn_fwd(ctypes.byref(_attn(b=0)), *[NULL] * 8, 0, NULL) == 0


def test_attn_step_arguments():
    lib = _lib.load()
    one = ctypes.byref(_attn(s=1, valid_len=1))
    assert lib.moments_attn_step(ctypes.byref(_attn()), *[FAKE] * 5, 8, FAKE, FAKE, NULL) == -1      # s != 1
    assert lib.moments_attn_step(one, *[FAKE] * 4, NULL, 1, FAKE, FAKE, NULL) == -1                   # pool below b
    assert lib.moments_attn_step(one, *[FAKE] * 5, -1, FAKE, FAKE, NULL) == -1
    assert lib.moments_attn_step(one, *[FAKE] * 5, 8, NULL, FAKE, NULL) == -1
    assert lib.moments_attn_step(one, *[FAKE] * 5, 8, ODD, FAKE, NULL) == -1


def _qk(**kw):
    d = dict(b=2, s=5, c=1, h=4, g=2, r=16, q_stride=0, k_stride=0, rope_dim=8, quat_blocks=0, rot_h=4,
             dtype=_lib.F32, rot_kind=M.ROT_PAIRWISE, eps=1e-5, reserved=0)
    d.update(kw)
    return M.QkDesc(**d)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(rot_h=1), 0), (dict(q_stride=40), 0), (dict(s=0), 0), (dict(eps=0.0), 0),
    (dict(rot_kind=M.ROT_NONE, rope_dim=0), 0), (dict(rot_kind=M.ROT_QUAT, quat_blocks=4), 0),
    (dict(g=3), -1), (dict(rot_h=2), -1), (dict(q_stride=31), -1), (dict(k_stride=-5), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(rope_dim=7), -1), (dict(rope_dim=18), -1), (dict(rope_dim=0), -1),
    (dict(rot_kind=M.ROT_HALF, r=15), -1), (dict(rot_kind=M.ROT_QUAT, quat_blocks=5), -1),
    (dict(rot_kind=8), -1), (dict(dtype=3), -1),
    (dict(r=129), -2), (dict(c=5), -2), (dict(h=1000, g=2, rot_h=1), -2),
])
def test_qk_descriptor(kw, code):
    n = _lib.load().moments_qk_workspace_size(ctypes.byref(_qk(**kw)))
    assert (n > 0) if code == 0 else (n == code)


@pytest.mark.parametrize("kw,code", [
    (dict(rot_kind=M.ROT_QUAT, rope_dim=0, quat_blocks=2 ** 62), -1),        # four times it is zero in 64 bits
    (dict(c=2 ** 62), -2), (dict(r=2 ** 62), -2), (dict(b=2 ** 40, s=2 ** 40), -2),
])
def test_qk_sizes_that_would_wrap(kw, code):
    assert _lib.load().moments_qk_workspace_size(ctypes.byref(_qk(**kw))) == code


def test_qk_pointers():
    lib = _lib.load()
    d = ctypes.byref(_qk())
    ok = [FAKE] * 9
    for i in (0, 1, 2, 3, 6, 7, 8):
        bad = list(ok)
        bad[i] = NULL
        assert lib.moments_qk_fwd(d, *bad, NULL) == -1
    plain = ctypes.byref(_qk(rot_kind=M.ROT_NONE, rope_dim=0))
    assert lib.moments_qk_fwd(plain, *ok, NULL) == -1                        # rot without a rotation
    args = [FAKE] * 16
    assert lib.moments_qk_bwd(d, *args, FAKE, 16, NULL) == -3
    no_bias = list(args)
    no_bias[4] = NULL
    assert lib.moments_qk_bwd(d, *no_bias, FAKE, BIG, NULL) == -1            # d_bq without bq


def _tensors(dt=torch.float32):
    return dict(xhat=torch.zeros(2, 6, 1, 4, 8, dtype=dt), bhat=torch.zeros(2, 6, 1, 2, 16, dtype=dt),
                qhat=torch.zeros(2, 6, 1, 2, 16, dtype=dt), da=torch.zeros(2, 6, 4, dtype=dt), h0=None)


@pytest.mark.parametrize("name,bad,match", [
    ("bhat", torch.zeros(2, 6, 1, 2, 15), "bhat has shape"),
    ("qhat", torch.zeros(2, 6, 1, 4, 16), "qhat has shape"),
    ("da", torch.zeros(2, 6, 3), "da has shape"),
    ("da", torch.zeros(2, 6, 4, dtype=torch.float64), "dtype"),
    ("h0", torch.zeros(2, 4, 8, 16, dtype=torch.bfloat16), "h0 has dtype"),
    ("xhat", torch.zeros(6, 2, 1, 4, 8).transpose(0, 1), "contiguous"),
    ("h0", None, "GPU"),                     # everything right, but on the host
])
def test_attn_binding(name, bad, match):
    t = _tensors()
    d = M.attn_desc(t["xhat"], t["bhat"])
    t[name] = bad
    with pytest.raises(ValueError, match=match):
        M.moments_attn_fwd(d, **t)


def test_attn_binding_of_step_and_backward():
    t = _tensors()
    d = M.attn_desc(t["xhat"], t["bhat"])
    a = (t["xhat"], t["bhat"], t["qhat"], t["da"])
    with pytest.raises(ValueError, match="state has dtype"):
        M.moments_attn_step(d, *a, torch.zeros(2, 4, 8, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="slots has dtype"):
        M.moments_attn_step(d, *a, torch.zeros(2, 4, 8, 16), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="d_y has shape"):
        M.moments_attn_bwd(d, *a, None, torch.zeros(2, 6, 4, 8))
    with pytest.raises(ValueError, match="saved is required"):
        M.moments_attn_bwd_saved(d, *a, None, None, t["xhat"])
    with pytest.raises(ValueError, match="valid_lens"):
        M.attn_desc(t["xhat"], t["bhat"], valid_lens=torch.zeros(2, dtype=torch.int64))


def test_qk_binding():
    wide = torch.zeros(2, 5, 100)
    q = wide[:, :, :32].view(2, 5, 1, 2, 16)
    k = torch.zeros(2, 5, 1, 2, 16)
    w, rot = torch.zeros(16), torch.zeros(2, 5, 1, 4)
    d = M.qk_desc(q, k, 4, M.ROT_PAIRWISE, rot=rot)
    assert (d.q_stride, d.k_stride, d.rope_dim, d.rot_h) == (100, 32, 8, 1)
    with pytest.raises(ValueError, match="another token stride"):
        M.moments_qk_fwd(d, k, k, w, w, None, None, rot)
    with pytest.raises(ValueError, match="rot has shape"):
        M.moments_qk_fwd(d, q, k, w, w, None, None, rot[..., :3])
    with pytest.raises(ValueError, match="bq has shape"):
        M.moments_qk_fwd(d, q, k, w, w, torch.zeros(2, 16), None, rot)
    with pytest.raises(ValueError, match="together"):
        M.qk_desc(torch.zeros(2, 5, 1, 16, 2).transpose(3, 4), k, 4, M.ROT_NONE)
    with pytest.raises(ValueError, match="together"):
        M.qk_desc(torch.zeros(5, 2, 1, 2, 16).transpose(0, 1), k, 4, M.ROT_NONE)
    with pytest.raises(ValueError, match="GPU"):
        M.moments_qk_fwd(d, q, k, w, w, None, None, rot)
