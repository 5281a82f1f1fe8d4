"""Edges of linear attention and of the norms with rotation that the host decides:
what an empty call may leave out, layouts, sizes. No GPU is touched."""
import ctypes

from mamba_ssm_chunkwise_amd import _lib
from test_attn_abi import BIG, FAKE, NULL, _qk


def test_norm_gradients_of_no_tokens_launch_nothing():
    """s = 0 with every input and gradient absent: a call without work, in which no weights are read."""
    lib = _lib.load()
    d = ctypes.byref(_qk(s=0))
    assert lib.moments_qk_bwd(d, *[NULL] * 16, FAKE, BIG, NULL) == 0
