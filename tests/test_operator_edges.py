"""Edges of linear attention and of the norms with rotation that the host decides:
what an empty call may leave out, layouts, sizes. No GPU is touched."""
import ctypes

import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from mamba_ssm_chunkwise_amd import _lib
from test_attn_abi import BIG, FAKE, NULL, _attn, _qk


def test_norm_gradients_of_no_tokens_launch_nothing():
    """s = 0 with every input and gradient absent: a call without work, in which no weights are read."""
    lib = _lib.load()
    d = ctypes.byref(_qk(s=0))
    assert lib.moments_qk_bwd(d, *[NULL] * 16, FAKE, BIG, NULL) == 0


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("kind", ["transposed", "expanded", "strided"])
def test_one_token_of_another_layout_is_refused(which, kind):
    """One token (b = s = 1) under a descriptor made earlier, as decoding has it: its values have to lie
    together there too."""
    t = {n: torch.zeros(1, 1, 1, 2, 16) for n in ("q", "k")}
    w = torch.zeros(16)
    d = M.qk_desc(t["q"], t["k"], 4, M.ROT_NONE)
    t[which] = {"transposed": torch.zeros(1, 1, 1, 16, 2).transpose(3, 4),
                "expanded": torch.zeros(1, 1, 1, 1, 16).expand(1, 1, 1, 2, 16),
                "strided": torch.zeros(1, 1, 1, 2, 32)[..., ::2]}[kind]
    with pytest.raises(ValueError, match=f"{which} must hold each token's values together"):
        M.moments_qk_fwd(d, t["q"], t["k"], w, w)
    hat = torch.zeros(1, 1, 1, 4, 16)
    with pytest.raises(ValueError, match=f"{which} must hold each token's values together"):
        M.moments_qk_bwd(d, t["q"], t["k"], w, w, None, None, None, hat, hat)


def test_one_token_cut_out_of_a_projection_is_taken():
    """Any step to a next token that is not there: the checks pass as far as the device."""
    q = torch.zeros(1, 1, 100)[:, :, :32].view(1, 1, 1, 2, 16)
    d = M.qk_desc(torch.zeros(1, 1, 1, 2, 16), q, 4, M.ROT_NONE)
    w = torch.zeros(16)
    with pytest.raises(ValueError, match="GPU"):
        M.moments_qk_fwd(d, q, q, w, w)


@pytest.mark.parametrize("p", [1, 64, 65])
@pytest.mark.parametrize("chains,fwd,bwd", [(2 ** 22 - 1, 0, 0), (2 ** 22, 0, 0), (2 ** 23 - 1, 0, 0), (2 ** 23, 0, -2),
                                            (2 ** 24 - 1, 0, -2), (2 ** 24, -2, -2)])
def test_sizes_that_a_launch_cannot_hold(p, chains, fwd, bwd):
    """2^32 threads and more: 256 for each 64 state rows of a chain forwards, 512 for the gradients."""
    if p > 64:      # two workgroups a chain
        fwd, bwd = (0 if 2 * chains < 2 ** 24 else -2), (0 if 2 * chains < 2 ** 23 else -2)
    d = ctypes.byref(_attn(b=chains, h=1, g=1, s=1, p=p, r=1, valid_len=1))
    lib = _lib.load()
    assert lib.moments_attn_validate(d) == fwd
    for n, code in ((lib.moments_attn_workspace_size(d, 0), fwd), (lib.moments_attn_saved_size(d), fwd),
                    (lib.moments_attn_workspace_size(d, 1), bwd)):
        assert (n >= 0) if code == 0 else (n == code)
    if bwd != 0:
        assert lib.moments_attn_bwd(d, *[FAKE] * 12, FAKE, BIG, NULL) == bwd
        assert lib.moments_attn_bwd_saved(d, *[FAKE] * 5, FAKE, BIG, *[FAKE] * 7, FAKE, BIG, NULL) == bwd
    if fwd != 0:
        assert lib.moments_attn_fwd(d, *[FAKE] * 7, FAKE, BIG, NULL) == fwd
        assert lib.moments_attn_step(d, *[FAKE] * 5, chains, FAKE, FAKE, NULL) == fwd


def test_queries_between_elements_are_refused():
    lib, d = _lib.load(), ctypes.byref(_qk())
    for at, code in ((2, -1), (1, -1)):
        args = [ctypes.c_void_p((1 << 20) + at)] + [FAKE] * 8
        assert lib.moments_qk_fwd(d, *args, NULL) == code
        assert lib.moments_qk_fwd(d, FAKE, args[0], *[FAKE] * 7, NULL) == code
    for i in range(2, 9):      # all the others start at 16 bytes
        args = [FAKE] * 9
        args[i] = ctypes.c_void_p((1 << 20) + 8)
        assert lib.moments_qk_fwd(d, *args, NULL) == -1


@pytest.mark.parametrize("s", [5, 64, 5000])
def test_the_finite_check_does_not_change_the_workspace(monkeypatch, s):
    """A workspace sized before MOMENTS_CHECK_FINITE is set holds for the calls after it."""
    lib, d = _lib.load(), ctypes.byref(_attn(b=1, h=1, g=1, s=s, valid_len=s))
    sizes = lambda: [lib.moments_attn_workspace_size(d, i) for i in (0, 1)]  # noqa: E731
    monkeypatch.delenv("MOMENTS_CHECK_FINITE", raising=False)
    before = sizes()
    monkeypatch.setenv("MOMENTS_CHECK_FINITE", "1")
    assert sizes() == before
