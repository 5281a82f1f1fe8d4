"""Edges of the binding and of the C entry points of the gated recurrence, layer norm and the
gradients' norm and clipping, on the host. No GPU is touched."""
import contextlib
import inspect
import re

import pytest
import torch

import mamba_ssm_chunkwise_amd as M
from mamba_ssm_chunkwise_amd import _lib


def test_a_call_runs_on_its_tensors_device(monkeypatch):
    """HIP launches on the current device: tensors of another make theirs current for the call, on
    their own stream, and the one before is current again, after an error too."""
    now = [0]

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        try:
            yield
        finally:
            now[0] = before

    monkeypatch.setattr(M, "_current_device", lambda: now[0])
    monkeypatch.setattr(M, "_stream_of", lambda dev: 100 + dev.index)
    monkeypatch.setattr(torch.cuda, "device", device)
    seen = []

    def call(*args):
        seen.append((now[0], args))
        return args[0]

    for index in (0, 1, 3):
        M._launch(torch.device("cuda", index), call, 0, "a")
        assert seen[-1] == (index, (0, "a", 100 + index)) and now[0] == 0
        with pytest.raises(M.MomentsError):
            M._launch(torch.device("cuda", index), call, _lib.EINVAL)
        assert now[0] == 0


def test_every_launch_names_its_device():
    """No entry point that takes a stream is called in another way."""
    src = inspect.getsource(M)
    direct = set(re.findall(r"(?:lib|load\(\))\.(moments_\w+)\(", src))
    assert direct and all(re.search(r"_(size|validate|len|enable|reset|read)$", n) for n in direct), direct
    launched = set(re.findall(r"_launch\(dev, (?:lib|_lib\.load\(\))\.(moments_\w+),", src))
    takes_stream = {n for n in _lib.EXPORTS if re.search(r"_(fwd|bwd|step|norm|clip|static|save|saved)$", n)}
    assert launched == takes_stream


@pytest.mark.parametrize("s,stride,code", [
    (1, (1 << 25) + 8, 0), (1, 1 << 37, 0), (1, (1 << 37) + 1, -2), (2, 1 << 25, 0), (2, (1 << 25) + 1, -2),
    (0, (1 << 25) + 8, 0),
])
def test_strides_of_single_tokens(s, stride, code):
    """One token of each sequence may stand as far from the next's as a long projection is."""
    for which in ("x_stride", "g_stride", "z_stride"):
        d = M.RecDesc(b=3, s=s, w=16, valid_len=s, dtype=_lib.BF16, gate=1, has_z=1, **{which: stride})
        assert M.moments_rec_validate(d) == code, which


def test_gradients_from_an_iterator():
    """As a program writes them: the gradients of the parameters that have one."""
    layer = torch.nn.Linear(3, 4)
    layer(torch.ones(2, 3)).sum().backward()
    d = M.grad_desc(p.grad for p in layer.parameters() if p.grad is not None)
    assert d.count == 2 and d.in_place and [id(t) for t in d.out] == [id(p.grad) for p in layer.parameters()]
    out = [torch.empty(4, 3), torch.empty(4)]
    d = M.grad_desc((p.grad for p in layer.parameters()), out=iter(out))
    assert d.count == 2 and not d.in_place and d.out[0] is out[0] and d.out[1] is out[1]


def test_a_misaligned_gradient_is_not_called_an_overlap():
    raw = bytearray(64)
    odd = torch.frombuffer(raw, dtype=torch.float32, count=4, offset=2)
    g = torch.zeros(4)
    assert odd.data_ptr() % 4 == 2
    with pytest.raises(ValueError, match=r"grads\[1\] starts"):
        M.grad_desc([g, odd])
    with pytest.raises(ValueError, match=r"out\[0\] starts"):
        M.grad_desc([g], out=[odd])
    with pytest.raises(ValueError, match="overlap"):
        M.grad_desc([g, g])
