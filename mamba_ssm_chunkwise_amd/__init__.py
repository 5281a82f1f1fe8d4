"""MI355X-native physical-frame state moments (Mamba-3): fwd + recompute bwd.

Python entry points with the C ABI's names. They marshal torch tensors into the
HIP library (libmoments.so) and run on torch's current HIP stream of the tensors'
device, whichever device is current; no computation happens in Python. See include/moments.h for the operation.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import (BF16, F32, GATE_LOG, GATE_MIX, GATE_UNIT, ROT_HALF, ROT_NONE, ROT_PAIRWISE,  # noqa: F401
                   ROT_QUAT, AttnDesc, Desc, LnDesc, MomentsError, QkDesc, RecDesc)

__all__ = ["make_desc", "set_valid_lens", "moments_validate", "moments_workspace_size", "moments_fwd", "moments_fwd_static",
           "moments_bwd", "moments_saved_size", "moments_fwd_save", "moments_bwd_saved", "rot_desc", "moments_rot_workspace_size", "moments_rot_fwd", "moments_rot_bwd",
           "kernel_chunk_len",
           "attn_desc", "moments_attn_validate", "moments_attn_workspace_size", "moments_attn_saved_size",
           "moments_attn_fwd", "moments_attn_fwd_save", "moments_attn_bwd", "moments_attn_bwd_saved",
           "moments_attn_step", "qk_desc", "moments_qk_workspace_size", "moments_qk_fwd", "moments_qk_bwd",
           "rec_desc", "moments_rec_validate", "moments_rec_workspace_size", "moments_rec_saved_size",
           "moments_rec_fwd", "moments_rec_fwd_save", "moments_rec_bwd", "moments_rec_bwd_saved", "moments_rec_step",
           "ln_desc", "moments_ln_workspace_size", "moments_ln_fwd", "moments_ln_bwd",
           "grad_desc", "moments_grad_workspace_size", "moments_grad_norm", "moments_grad_clip",
           "AttnDesc", "QkDesc", "RecDesc", "LnDesc", "GradDesc", "GATE_LOG", "GATE_MIX", "GATE_UNIT",
           "Desc", "MomentsError", "ROT_NONE", "ROT_PAIRWISE", "ROT_HALF", "ROT_QUAT"]


def make_desc(xhat, bhat, chunk_len, valid_len, rot_kind, rope_dim=0, quat_blocks=0, dtype=None,
              valid_lens=None):
    b, s, c, h, p = xhat.shape
    r = bhat.shape[-1]
    if dtype is None:
        dtype = BF16 if xhat.dtype == torch.bfloat16 else F32
    d = Desc(b, s, c, h, p, r, int(chunk_len), int(valid_len), int(dtype), int(rot_kind),
             int(rope_dim), int(quat_blocks))
    return set_valid_lens(d, valid_lens)


def set_valid_lens(desc, valid_lens):
    """Per-sequence valid lengths: ``valid_lens`` is an int32 GPU tensor of shape
    [b] (or None for one length, desc.valid_len, for the whole batch). Sequence
    bi then uses min(max(valid_lens[bi], 0), desc.valid_len, s). The descriptor
    keeps a reference to the tensor, whose contents the kernels read."""
    if valid_lens is None:
        desc.valid_lens = None
        desc._valid_lens_ref = None
        return desc
    if not isinstance(valid_lens, torch.Tensor):
        raise ValueError("valid_lens must be a torch.Tensor")
    if tuple(valid_lens.shape) != (int(desc.b),) or valid_lens.dtype != torch.int32:
        raise ValueError(f"valid_lens must be int32 of shape ({desc.b},), got {valid_lens.dtype} "
                         f"{tuple(valid_lens.shape)}")
    if valid_lens.device.type != "cuda" or not valid_lens.is_contiguous():
        raise ValueError("valid_lens must be a contiguous GPU tensor")
    desc.valid_lens = valid_lens.data_ptr()
    desc._valid_lens_ref = valid_lens
    return desc


def moments_validate(desc: Desc) -> int:
    return _lib.load().moments_validate(ctypes.byref(desc))


def moments_workspace_size(desc: Desc, is_bwd: bool) -> int:
    n = _lib.load().moments_workspace_size(ctypes.byref(desc), int(bool(is_bwd)))
    if n < 0:
        _lib.check(int(n))
    return int(n)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _expect(name, t, shape, dtype, device, optional=False):
    """Raises ValueError unless t is a contiguous tensor of exactly this shape and
    dtype on this device (the kernels index every buffer from the descriptor)."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, the descriptor needs {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, the descriptor needs {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _input_specs(desc: Desc):
    """Expected shapes and dtype of the five inputs (rot: None when there is no rotation)."""
    b, s, c, h, p, r = desc.b, desc.s, desc.c, desc.h, desc.p, desc.r
    if desc.rot_kind in (ROT_PAIRWISE, ROT_HALF):
        rot = (b, s, h, desc.rope_dim // 2)
    elif desc.rot_kind == ROT_QUAT:
        rot = (b, s, h, desc.quat_blocks, 4)
    else:
        rot = None
    dt = torch.bfloat16 if desc.dtype == BF16 else torch.float32
    return {"xhat": (b, s, c, h, p), "bhat": (b, s, c, h, r), "da": (b, s, h), "rot": rot,
            "h0": (b, h, p, r)}, dt


def _check_inputs(desc: Desc, xhat, bhat, da, rot, h0):
    """Shapes, dtypes and devices of the inputs against the descriptor (all on
    xhat's device, which must be a GPU)."""
    if not isinstance(xhat, torch.Tensor):
        raise ValueError("xhat must be a torch.Tensor")
    dev = xhat.device
    if desc.valid_lens:
        ref = getattr(desc, "_valid_lens_ref", None)
        if ref is None or ref.data_ptr() != desc.valid_lens:
            raise ValueError("set per-sequence lengths with set_valid_lens (the descriptor keeps the tensor)")
        if ref.device != dev:
            raise ValueError(f"valid_lens is on {ref.device}, the inputs on {dev}")
    specs, dt = _input_specs(desc)
    _expect("xhat", xhat, specs["xhat"], dt, dev)
    _expect("bhat", bhat, specs["bhat"], dt, dev)
    _expect("da", da, specs["da"], dt, dev)
    if specs["rot"] is None:
        if rot is not None:
            raise ValueError("rot must be None when the descriptor has no rotation")
    else:
        _expect("rot", rot, specs["rot"], dt, dev)
    _expect("h0", h0, specs["h0"], dt, dev, optional=True)
    return dev, specs, dt


def _require_gpu(dev):
    if dev.type != "cuda":
        raise ValueError(f"the inputs are on {dev}; the kernels need GPU tensors")
    _lib.load()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(dev):
    """torch's current stream on dev as an integer handle."""
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _launch(dev, call, *args):
    """Calls the library with torch's current stream on dev as the last argument and raises on
    an error. HIP launches on the current device, so dev is made that for the call."""
    if dev.index is None or dev.index == _current_device():
        rc = call(*args, _stream_of(dev))
    else:
        with torch.cuda.device(dev.index):
            rc = call(*args, _stream_of(dev))
    _lib.check(rc)


def _workspace(desc, is_bwd, device, workspace):
    n = moments_workspace_size(desc, is_bwd)
    if workspace is None:
        return torch.empty(max(n, 1), dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    if workspace.numel() * workspace.element_size() < n:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, "
                         f"the descriptor needs {n}")
    return workspace


def moments_fwd(desc: Desc, xhat, bhat, da, rot, h0, m2=None, m1=None, workspace=None):
    """Returns (m2 [b,h,r,r], m1 [b,h,p,r]) float32."""
    dev, _, _ = _check_inputs(desc, xhat, bhat, da, rot, h0)
    _expect("m2", m2, (desc.b, desc.h, desc.r, desc.r), torch.float32, dev, optional=True)
    _expect("m1", m1, (desc.b, desc.h, desc.p, desc.r), torch.float32, dev, optional=True)
    _require_gpu(dev)
    if m2 is None:
        m2 = torch.empty(desc.b, desc.h, desc.r, desc.r, dtype=torch.float32, device=dev)
    if m1 is None:
        m1 = torch.empty(desc.b, desc.h, desc.p, desc.r, dtype=torch.float32, device=dev)
    ws = _workspace(desc, False, dev, workspace)
    _launch(dev, _lib.load().moments_fwd, ctypes.byref(desc), _ptr(xhat), _ptr(bhat), _ptr(da), _ptr(rot), _ptr(h0),
            _ptr(m2), _ptr(m1), _ptr(ws), ws.numel() * ws.element_size())
    return m2, m1


def moments_fwd_static(desc: Desc, xhat, bhat, da, rot, h0, m2, m1):
    """moments_fwd without a workspace: the library's static device scratch
    (64 MiB per GPU) holds the kernels' intermediates. m2 and m1 are the
    caller's float32 output tensors; nothing is allocated here."""
    dev, _, _ = _check_inputs(desc, xhat, bhat, da, rot, h0)
    _expect("m2", m2, (desc.b, desc.h, desc.r, desc.r), torch.float32, dev)
    _expect("m1", m1, (desc.b, desc.h, desc.p, desc.r), torch.float32, dev)
    _require_gpu(dev)
    _launch(dev, _lib.load().moments_fwd_static, ctypes.byref(desc), _ptr(xhat), _ptr(bhat), _ptr(da), _ptr(rot),
            _ptr(h0), _ptr(m2), _ptr(m1))
    return m2, m1


def moments_saved_size(desc: Desc) -> int:
    """Bytes of the saved-carry buffer of moments_fwd_save / moments_bwd_saved."""
    n = _lib.load().moments_saved_size(ctypes.byref(desc))
    if n < 0:
        _lib.check(int(n))
    return int(n)


def _saved_buffer(desc, device, saved):
    n = moments_saved_size(desc)
    if saved is None:
        return torch.empty(max(n, 1), dtype=torch.uint8, device=device)
    if not isinstance(saved, torch.Tensor) or saved.device != device or not saved.is_contiguous():
        raise ValueError(f"saved must be a contiguous tensor on {device}")
    if saved.numel() * saved.element_size() < n:
        raise ValueError(f"saved holds {saved.numel() * saved.element_size()} bytes, the descriptor needs {n}")
    return saved


def moments_fwd_save(desc: Desc, xhat, bhat, da, rot, h0, m2=None, m1=None, saved=None, workspace=None):
    """moments_fwd that also keeps the chunk-boundary states for the backward.
    Returns (m2, m1, saved); saved is an opaque uint8 device tensor to pass to
    moments_bwd_saved with the same descriptor and inputs."""
    dev, _, _ = _check_inputs(desc, xhat, bhat, da, rot, h0)
    _expect("m2", m2, (desc.b, desc.h, desc.r, desc.r), torch.float32, dev, optional=True)
    _expect("m1", m1, (desc.b, desc.h, desc.p, desc.r), torch.float32, dev, optional=True)
    _require_gpu(dev)
    if m2 is None:
        m2 = torch.empty(desc.b, desc.h, desc.r, desc.r, dtype=torch.float32, device=dev)
    if m1 is None:
        m1 = torch.empty(desc.b, desc.h, desc.p, desc.r, dtype=torch.float32, device=dev)
    sv = _saved_buffer(desc, dev, saved)
    ws = _workspace(desc, False, dev, workspace)
    _launch(dev, _lib.load().moments_fwd_save, ctypes.byref(desc), _ptr(xhat), _ptr(bhat), _ptr(da), _ptr(rot),
            _ptr(h0), _ptr(m2), _ptr(m1), _ptr(sv), sv.numel(), _ptr(ws), ws.numel() * ws.element_size())
    return m2, m1, sv


def moments_bwd_saved(desc: Desc, xhat, bhat, da, rot, h0, saved, d_m2, d_m1,
                      want=("xhat", "bhat", "da", "rot", "h0"), out=None, workspace=None):
    """moments_bwd reading the chunk-boundary states moments_fwd_save kept
    (no carry pass). Same returns as moments_bwd."""
    return moments_bwd(desc, xhat, bhat, da, rot, h0, d_m2, d_m1, want=want, out=out, workspace=workspace,
                       _saved=saved)


def moments_bwd(desc: Desc, xhat, bhat, da, rot, h0, d_m2, d_m1, want=("xhat", "bhat", "da", "rot", "h0"),
                out=None, workspace=None, _saved=None):
    """Returns dict d_xhat, d_bhat, d_da, d_rot, d_h0 (input dtype; None when
    not wanted or not defined)."""
    dev, specs, dt = _check_inputs(desc, xhat, bhat, da, rot, h0)
    _expect("d_m2", d_m2, (desc.b, desc.h, desc.r, desc.r), torch.float32, dev)
    _expect("d_m1", d_m1, (desc.b, desc.h, desc.p, desc.r), torch.float32, dev)
    out = dict(out or {})
    for k in ("xhat", "bhat", "da", "rot", "h0"):
        key = "d_" + k
        if k in want and specs[k] is not None:
            _expect(key, out.get(key), specs[k], dt, dev, optional=True)
        else:
            out[key] = None
    _require_gpu(dev)
    for k in ("xhat", "bhat", "da", "rot", "h0"):
        key = "d_" + k
        if k in want and specs[k] is not None and out.get(key) is None:
            out[key] = torch.empty(specs[k], dtype=dt, device=dev)
    ws = _workspace(desc, True, dev, workspace)
    grads = (_ptr(d_m2), _ptr(d_m1), _ptr(out["d_xhat"]), _ptr(out["d_bhat"]), _ptr(out["d_da"]),
             _ptr(out["d_rot"]), _ptr(out["d_h0"]), _ptr(ws), ws.numel() * ws.element_size())
    ins = (ctypes.byref(desc), _ptr(xhat), _ptr(bhat), _ptr(da), _ptr(rot), _ptr(h0))
    if _saved is None:
        _launch(dev, _lib.load().moments_bwd, *ins, *grads)
    else:
        sv = _saved_buffer(desc, dev, _saved)
        _launch(dev, _lib.load().moments_bwd_saved, *ins, _ptr(sv), sv.numel() * sv.element_size(), *grads)
    return out


def rot_desc(inc, rot_kind, rope_dim=0, quat_blocks=0):
    """Descriptor of the rotation-sequence producer for increments ``inc``
    ([b,s,h,a] angles with rope_dim = 2a, or [b,s,h,J,4] quaternions). Only b,
    s, h, dtype, rot_kind and rope_dim / quat_blocks are read by the library."""
    if not isinstance(inc, torch.Tensor):
        raise ValueError("inc must be a torch.Tensor")
    b, s, h = (int(x) for x in inc.shape[:3])
    if rot_kind == ROT_QUAT and quat_blocks == 0 and inc.dim() == 5:
        quat_blocks = int(inc.shape[3])
    if rot_kind in (ROT_PAIRWISE, ROT_HALF) and rope_dim == 0 and inc.dim() == 4:
        rope_dim = 2 * int(inc.shape[3])
    dtype = BF16 if inc.dtype == torch.bfloat16 else F32
    return Desc(b, s, 1, h, 1, 1, 1, s, int(dtype), int(rot_kind), int(rope_dim), int(quat_blocks))


def _rot_shape(desc: Desc):
    if desc.rot_kind == ROT_QUAT:
        return (desc.b, desc.s, desc.h, desc.quat_blocks, 4)
    if desc.rot_kind in (ROT_PAIRWISE, ROT_HALF):
        return (desc.b, desc.s, desc.h, desc.rope_dim // 2)
    raise ValueError("the producer needs a rotation (rot_kind must not be ROT_NONE)")


def moments_rot_workspace_size(desc: Desc, is_bwd: bool) -> int:
    n = _lib.load().moments_rot_workspace_size(ctypes.byref(desc), int(bool(is_bwd)))
    if n < 0:
        _lib.check(int(n))
    return int(n)


def _rot_call(desc, is_bwd, inc, d_rot, out):
    if not isinstance(inc, torch.Tensor):
        raise ValueError("inc must be a torch.Tensor")
    dev = inc.device
    shape = _rot_shape(desc)
    dt = torch.bfloat16 if desc.dtype == BF16 else torch.float32
    _expect("inc", inc, shape, dt, dev)
    if is_bwd:
        _expect("d_rot", d_rot, shape, dt, dev)
    _expect("out", out, shape, dt, dev, optional=True)
    _require_gpu(dev)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
    n = moments_rot_workspace_size(desc, is_bwd)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    lib = _lib.load()
    if is_bwd:
        _launch(dev, lib.moments_rot_bwd, ctypes.byref(desc), _ptr(inc), _ptr(d_rot), _ptr(out), _ptr(ws), n)
    else:
        _launch(dev, lib.moments_rot_fwd, ctypes.byref(desc), _ptr(inc), _ptr(out), _ptr(ws), n)
    return out


def moments_rot_fwd(desc: Desc, inc, rot=None):
    """Cumulative rotation (the moments path's ``rot``) from per-token increments."""
    return _rot_call(desc, False, inc, None, rot)


def moments_rot_bwd(desc: Desc, inc, d_rot, d_inc=None):
    """Cotangent of the increments from the cotangent of the cumulative rotation."""
    return _rot_call(desc, True, inc, d_rot, d_inc)


# ---------------------------------------------------------------- linear attention
# These entry points also serve single tokens, where the host's time counts: tensors are
# checked in one pass and pointers go to the library as plain integers.
_DTYPES = {F32: torch.float32, BF16: torch.bfloat16}


def _tensors_ok(dev, specs):
    """Checks (name, tensor, shape, dtype, optional) each as _expect does; returns the
    tensors' addresses (None for an absent optional one)."""
    out = []
    at = -1 if dev.index is None else dev.index
    for name, t, shape, dtype, optional in specs:
        if t is None and optional:
            out.append(None)
        elif (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.get_device() == at
              and t.is_contiguous() and (at >= 0 or t.device == dev)):
            out.append(t.data_ptr())
        else:
            _expect(name, t, shape, dtype, dev)   # names what is wrong
            out.append(t.data_ptr())
    return out


def _gpu(dev):
    if dev.type != "cuda":
        raise ValueError(f"the inputs are on {dev}; the kernels need GPU tensors")
    return _lib.load()


def _buffer(name, n, device, t):
    """The caller's scratch tensor, checked, or a new one of n bytes (None for none)."""
    if t is None:
        return torch.empty(n, dtype=torch.uint8, device=device) if n else None
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    if t.numel() * t.element_size() < n:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, the descriptor needs {n}")
    return t


def _scratch(t):
    """(address, bytes) of a scratch tensor or None."""
    return (None, 0) if t is None else (t.data_ptr(), t.numel() * t.element_size())


def _wrote(*tensors):
    """Tells autograd that the library wrote to these tensors of the caller's."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None])


def _size(n):
    if n < 0:
        _lib.check(int(n))
    return int(n)


def _shape5(name, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 5:
        raise ValueError(f"{name} must be a torch.Tensor of five dimensions")
    return t.shape


def attn_desc(xhat, bhat, valid_len=None, valid_lens=None, dtype=None) -> AttnDesc:
    """Descriptor of linear attention for xhat [b,s,c,h,p] and keys bhat
    [b,s,c,g,r] of g groups of heads. ``valid_len`` defaults to s; ``valid_lens``
    as in make_desc."""
    b, s, c, h, p = _shape5("xhat", xhat)
    _, _, _, g, r = _shape5("bhat", bhat)
    if dtype is None:
        dtype = BF16 if xhat.dtype is torch.bfloat16 else F32
    d = AttnDesc(b, s, c, h, g, p, r, s if valid_len is None else int(valid_len), int(dtype))
    return set_valid_lens(d, valid_lens) if valid_lens is not None else d


def moments_attn_validate(desc: AttnDesc) -> int:
    return _lib.load().moments_attn_validate(ctypes.byref(desc))


def moments_attn_workspace_size(desc: AttnDesc, is_bwd: bool) -> int:
    return _size(_lib.load().moments_attn_workspace_size(ctypes.byref(desc), int(bool(is_bwd))))


def moments_attn_saved_size(desc: AttnDesc) -> int:
    """Bytes of the buffer of moments_attn_fwd_save / moments_attn_bwd_saved."""
    return _size(_lib.load().moments_attn_saved_size(ctypes.byref(desc)))


def _attn_inputs(desc: AttnDesc, xhat, bhat, qhat, da, h0):
    """Checks the inputs against the descriptor (all on xhat's device). Returns the
    device and their addresses."""
    if not isinstance(xhat, torch.Tensor):
        raise ValueError("xhat must be a torch.Tensor")
    dev, dt = xhat.device, _DTYPES.get(desc.dtype)
    if desc.valid_lens:
        ref = getattr(desc, "_valid_lens_ref", None)
        if ref is None or ref.data_ptr() != desc.valid_lens:
            raise ValueError("set per-sequence lengths with set_valid_lens (the descriptor keeps the tensor)")
        if ref.device != dev:
            raise ValueError(f"valid_lens is on {ref.device}, the inputs on {dev}")
    b, s, c, h, p = desc.b, desc.s, desc.c, desc.h, desc.p
    keys = (b, s, c, desc.g, desc.r)
    return dev, _tensors_ok(dev, (
        ("xhat", xhat, (b, s, c, h, p), dt, False), ("bhat", bhat, keys, dt, False), ("qhat", qhat, keys, dt, False),
        ("da", da, (b, s, h), dt, False), ("h0", h0, (b, h, p, desc.r), torch.float32, True)))


def _attn_forward(desc, xhat, bhat, qhat, da, h0, y, h_last, saved, want_saved, workspace):
    dev, ins = _attn_inputs(desc, xhat, bhat, qhat, da, h0)
    state = (desc.b, desc.h, desc.p, desc.r)
    if y is not None or h_last is not None:
        _tensors_ok(dev, (("y", y, xhat.shape, xhat.dtype, True), ("h_last", h_last, state, torch.float32, True)))
    lib = _gpu(dev)
    ws = _buffer("workspace", moments_attn_workspace_size(desc, False), dev, workspace)
    _wrote(y, h_last, saved)
    if y is None:
        y = torch.empty_like(xhat)
    if h_last is None:
        h_last = torch.empty(state, dtype=torch.float32, device=dev)
    head = (ctypes.byref(desc), *ins, y.data_ptr(), h_last.data_ptr())
    tail = _scratch(ws)
    if want_saved:
        saved = _buffer("saved", moments_attn_saved_size(desc), dev, saved)
        _launch(dev, lib.moments_attn_fwd_save, *head, *_scratch(saved), *tail)
        return y, h_last, torch.empty(0, dtype=torch.uint8, device=dev) if saved is None else saved
    _launch(dev, lib.moments_attn_fwd, *head, *tail)
    return y, h_last


def moments_attn_fwd(desc: AttnDesc, xhat, bhat, qhat, da, h0=None, y=None, h_last=None, workspace=None):
    """Linear attention over a whole sequence: returns (y [b,s,c,h,p] in the input
    dtype, h_last [b,h,p,r] float32)."""
    return _attn_forward(desc, xhat, bhat, qhat, da, h0, y, h_last, None, False, workspace)


def moments_attn_fwd_save(desc: AttnDesc, xhat, bhat, qhat, da, h0=None, y=None, h_last=None, saved=None,
                          workspace=None):
    """moments_attn_fwd that also keeps the states entering the kernels' chunks.
    Returns (y, h_last, saved); saved is opaque, for moments_attn_bwd_saved."""
    return _attn_forward(desc, xhat, bhat, qhat, da, h0, y, h_last, saved, True, workspace)


def _gradients(dev, want, out, like):
    """The dict of gradients d_<name> for the inputs in ``like``: the caller's tensors
    (checked) or new ones; None where not wanted or the input is absent."""
    out = dict(out or {})
    _tensors_ok(dev, [("d_" + k, out.get("d_" + k), t.shape, t.dtype, True) for k, t in like.items()
                      if k in want and t is not None])
    _gpu(dev)
    _wrote(*[out.get("d_" + k) for k, t in like.items() if k in want and t is not None])
    for k, t in like.items():
        if k not in want or t is None:
            out["d_" + k] = None
        elif out.get("d_" + k) is None:
            out["d_" + k] = torch.empty(t.shape, dtype=t.dtype, device=dev)
    return out, [None if out["d_" + k] is None else out["d_" + k].data_ptr() for k in like]


def moments_attn_bwd(desc: AttnDesc, xhat, bhat, qhat, da, h0, d_y, d_h_last=None,
                     want=("xhat", "bhat", "qhat", "da", "h0"), out=None, workspace=None, _saved=None):
    """Returns dict d_xhat, d_bhat, d_qhat, d_da (input dtype), d_h0 (float32); None
    when not wanted (d_h0: or when there is no h0)."""
    dev, ins = _attn_inputs(desc, xhat, bhat, qhat, da, h0)
    cot = _tensors_ok(dev, (("d_y", d_y, xhat.shape, xhat.dtype, False),
                            ("d_h_last", d_h_last, (desc.b, desc.h, desc.p, desc.r), torch.float32, True)))
    out, grads = _gradients(dev, want, out, {"xhat": xhat, "bhat": bhat, "qhat": qhat, "da": da, "h0": h0})
    lib = _lib.load()
    ws = _buffer("workspace", moments_attn_workspace_size(desc, True), dev, workspace)
    tail = (*cot, *grads, *_scratch(ws))
    if _saved is None:
        _launch(dev, lib.moments_attn_bwd, ctypes.byref(desc), *ins, *tail)
    else:
        sv = _buffer("saved", moments_attn_saved_size(desc), dev, _saved)
        _launch(dev, lib.moments_attn_bwd_saved, ctypes.byref(desc), *ins, *_scratch(sv), *tail)
    return out


def moments_attn_bwd_saved(desc: AttnDesc, xhat, bhat, qhat, da, h0, saved, d_y, d_h_last=None,
                           want=("xhat", "bhat", "qhat", "da", "h0"), out=None, workspace=None):
    """moments_attn_bwd reading what moments_attn_fwd_save kept. Same returns."""
    if saved is None:
        raise ValueError("saved is required")
    return moments_attn_bwd(desc, xhat, bhat, qhat, da, h0, d_y, d_h_last, want=want, out=out,
                            workspace=workspace, _saved=saved)


def moments_attn_step(desc: AttnDesc, xhat, bhat, qhat, da, state, slots=None, y=None):
    """One token of each sequence (s = 1) on a pool of states, state [nslots,h,p,r]
    float32, updated in place; ``slots`` int32 [b] (None: slot i for sequence i; a
    slot outside the pool marks an unused row, whose y is zero). Returns y."""
    dev, ins = _attn_inputs(desc, xhat, bhat, qhat, da, None)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a torch.Tensor [nslots,h,p,r]")
    n = state.shape[0]
    st, sl, out = _tensors_ok(dev, (("state", state, (n, desc.h, desc.p, desc.r), torch.float32, False),
                                    ("slots", slots, (desc.b,), torch.int32, True),
                                    ("y", y, xhat.shape, xhat.dtype, True)))
    lib = _gpu(dev)
    _wrote(state, y)
    if y is None:
        y = torch.empty_like(xhat)
        out = y.data_ptr()
    _launch(dev, lib.moments_attn_step, ctypes.byref(desc), *ins[:4], sl, n, st, out)
    return y


# ---------------------------------------------------------------- norms of queries and keys
def qk_desc(q, k, h, rot_kind, rot=None, eps=1e-5, rope_dim=None, quat_blocks=None) -> QkDesc:
    """Descriptor of the norms with rotation for q and k [b,s,c,g,r] and h heads.
    q and k may be columns of a wider projection: each token's values together,
    tokens a fixed stride apart. The rotated width and the heads of the rotation
    are taken from ``rot`` ([b,s,h or 1,a] angles or [b,s,h or 1,J,4])."""
    strides = [_token_stride("q", q), _token_stride("k", k)]
    b, s, c, g, r = q.shape
    rot_h = h
    if rot_kind != ROT_NONE:
        if not isinstance(rot, torch.Tensor) or rot.dim() != (5 if rot_kind == ROT_QUAT else 4):
            raise ValueError("rot must be a torch.Tensor [b,s,heads,a] of angles or [b,s,heads,J,4] of quaternions")
        rot_h = rot.shape[2]
        if rot_kind == ROT_QUAT:
            quat_blocks = rot.shape[3] if quat_blocks is None else quat_blocks
        else:
            rope_dim = 2 * rot.shape[3] if rope_dim is None else rope_dim
    return QkDesc(b, s, c, h, g, r, strides[0], strides[1], rope_dim or 0, quat_blocks or 0, rot_h,
                  BF16 if q.dtype is torch.bfloat16 else F32, int(rot_kind), float(eps))


def _token_stride(name, t):
    """Elements between tokens of t [b,s,c,g,r] (0 where any would do)."""
    b, s, c, g, r = _shape5(name, t)
    if t.is_contiguous():
        return c * g * r if b * s > 1 else 0
    if t.numel() == 0:
        return 0
    sb, ss, sc, sg, sr = t.stride()
    step = ss if s > 1 else (sb if b > 1 else c * g * r)
    inner = (r == 1 or sr == 1) and (g == 1 or sg == r) and (c == 1 or sc == g * r)
    if not inner or step < c * g * r or (b > 1 and s > 1 and sb != s * step):
        raise ValueError(f"{name} must hold each token's values together, tokens a fixed stride apart")
    return step


def _qk_inputs(desc: QkDesc, q, k, wq, wk, bq, bk, rot):
    """Checks the inputs against the descriptor; returns the device, the dtype and the
    inputs' addresses."""
    if not isinstance(q, torch.Tensor):
        raise ValueError("q must be a torch.Tensor")
    dev, dt = q.device, _DTYPES.get(desc.dtype)
    b, s, c, h, g, r = desc.b, desc.s, desc.c, desc.h, desc.g, desc.r
    row, raw = c * g * r, (b, s, c, g, r)
    for name, t, stride in (("q", q, desc.q_stride), ("k", k, desc.k_stride)):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch.Tensor")
        if t.shape != raw or t.dtype is not dt or t.device != dev:
            raise ValueError(f"{name} must be {dt} of shape {(b, s, c, g, r)} on {dev}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        step = _token_stride(name, t) or row   # also one token's values have to lie together
        if b * s > 1 and step != (stride or row):
            raise ValueError(f"{name} has another token stride than the descriptor ({stride or row})")
    f32, kind = torch.float32, desc.rot_kind
    specs = [("wq", wq, (r,), f32, False), ("wk", wk, (r,), f32, False), ("bq", bq, (h, r), f32, True),
             ("bk", bk, (h, r), f32, True)]
    if kind == ROT_NONE:
        if rot is not None:
            raise ValueError("rot must be None when the descriptor has no rotation")
    elif kind == ROT_QUAT:
        specs.append(("rot", rot, (b, s, desc.rot_h, desc.quat_blocks, 4), dt, False))
    else:
        specs.append(("rot", rot, (b, s, desc.rot_h, desc.rope_dim // 2), dt, False))
    ptrs = [q.data_ptr(), k.data_ptr(), *_tensors_ok(dev, specs)]
    return dev, dt, ptrs if kind != ROT_NONE else [*ptrs, None]


def moments_qk_workspace_size(desc: QkDesc) -> int:
    """Bytes of the backward's workspace (the forward needs none)."""
    return _size(_lib.load().moments_qk_workspace_size(ctypes.byref(desc)))


def moments_qk_fwd(desc: QkDesc, q, k, wq, wk, bq=None, bk=None, rot=None, qhat=None, khat=None):
    """Returns (qhat, khat) [b,s,c,h,r]: normed, weighted, biased and turned into the
    frame of the cached states (khat is what the moments path takes as bhat)."""
    dev, dt, ins = _qk_inputs(desc, q, k, wq, wk, bq, bk, rot)
    shape = (desc.b, desc.s, desc.c, desc.h, desc.r)
    if qhat is not None or khat is not None:
        _tensors_ok(dev, (("qhat", qhat, shape, dt, True), ("khat", khat, shape, dt, True)))
    lib = _gpu(dev)
    _wrote(qhat, khat)
    if qhat is None:
        qhat = torch.empty(shape, dtype=dt, device=dev)
    if khat is None:
        khat = torch.empty_like(qhat)
    _launch(dev, lib.moments_qk_fwd, ctypes.byref(desc), *ins, qhat.data_ptr(), khat.data_ptr())
    return qhat, khat


def moments_qk_bwd(desc: QkDesc, q, k, wq, wk, bq, bk, rot, d_qhat, d_khat,
                   want=("q", "k", "wq", "wk", "bq", "bk", "rot"), out=None, workspace=None):
    """Returns dict d_q, d_k, d_rot (input dtype, dense), d_wq, d_wk, d_bq, d_bk
    (float32); None when not wanted or not defined."""
    dev, dt, ins = _qk_inputs(desc, q, k, wq, wk, bq, bk, rot)
    shape = (desc.b, desc.s, desc.c, desc.h, desc.r)
    cot = _tensors_ok(dev, (("d_qhat", d_qhat, shape, dt, False), ("d_khat", d_khat, shape, dt, False)))
    out, grads = _gradients(dev, want, out, {"q": q, "k": k, "wq": wq, "wk": wk, "bq": bq, "bk": bk, "rot": rot})
    ws = _buffer("workspace", moments_qk_workspace_size(desc), dev, workspace)
    _launch(dev, _lib.load().moments_qk_bwd, ctypes.byref(desc), *ins, *cot, *grads, *_scratch(ws))
    return out


# ---------------------------------------------------------------- gated linear recurrence
def _dense_like(t):
    """An uninitialised dense tensor of t's shape and dtype."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _row_stride(name, t):
    """Elements between tokens of t [b,s,w] (0 where any would do)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a torch.Tensor of three dimensions")
    b, s, n = t.shape
    if t.numel() == 0 or (b * s == 1 and t.is_contiguous()):
        return 0
    sb, ss, sw = t.stride()
    step = ss if s > 1 else (sb if b > 1 else n)
    if (n > 1 and sw != 1) or step < n or (b > 1 and s > 1 and sb != s * step):
        raise ValueError(f"{name} must hold each token's values together, tokens a fixed stride apart")
    return step


def rec_desc(x, g, z=None, gate=GATE_LOG, valid_len=None, valid_lens=None) -> RecDesc:
    """Descriptor of the gated linear recurrence for x, g and (or None) z [b,s,w]; they
    may be columns of one projection: each token's values together, tokens a fixed stride
    apart. ``valid_len`` defaults to s; ``valid_lens`` as in make_desc."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a torch.Tensor [b,s,w]")
    b, s, w = x.shape
    dense, steps = (s * w, w, 1), []
    for name, t in (("x", x), ("g", g), ("z", z)):
        if t is None and name == "z":
            steps.append(0)
        else:   # dense rows are what most calls have
            steps.append(w if isinstance(t, torch.Tensor) and t.stride() == dense else _row_stride(name, t))
    d = RecDesc(b, s, w, s if valid_len is None else int(valid_len), *steps,
                BF16 if x.dtype is torch.bfloat16 else F32, int(gate), 0 if z is None else 1)
    return set_valid_lens(d, valid_lens) if valid_lens is not None else d


def moments_rec_validate(desc: RecDesc) -> int:
    return _lib.load().moments_rec_validate(ctypes.byref(desc))


def moments_rec_workspace_size(desc: RecDesc, is_bwd: bool) -> int:
    return _size(_lib.load().moments_rec_workspace_size(ctypes.byref(desc), int(bool(is_bwd))))


def moments_rec_saved_size(desc: RecDesc) -> int:
    """Bytes of the buffer of moments_rec_fwd_save / moments_rec_bwd_saved."""
    return _size(_lib.load().moments_rec_saved_size(ctypes.byref(desc)))


def _rec_inputs(desc: RecDesc, x, g, z, h0):
    """Checks the inputs against the descriptor (all on x's device). Returns the device
    and their addresses."""
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a torch.Tensor")
    dev, dt = x.device, _DTYPES.get(desc.dtype)
    if desc.valid_lens:
        ref = getattr(desc, "_valid_lens_ref", None)
        if ref is None or ref.data_ptr() != desc.valid_lens:
            raise ValueError("set per-sequence lengths with set_valid_lens (the descriptor keeps the tensor)")
        if ref.device != dev:
            raise ValueError(f"valid_lens is on {ref.device}, the inputs on {dev}")
    if (z is not None) != bool(desc.has_z):
        raise ValueError("z must be None when the descriptor has no z" if z is not None else "z is required")
    b, s, w = shape = (desc.b, desc.s, desc.w)
    at = -1 if dev.index is None else dev.index
    ptrs = []
    for name, t, stride in (("x", x, desc.x_stride), ("g", g, desc.g_stride), ("z", z, desc.z_stride)):
        if t is None and name == "z":
            ptrs.append(None)
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch.Tensor")
        if t.shape != shape or t.dtype is not dt or t.get_device() != at or (at < 0 and t.device != dev):
            raise ValueError(f"{name} must be {dt} of shape {shape} on {dev}, got {t.dtype} {tuple(t.shape)} "
                             f"on {t.device}")
        step = stride or w
        # also one token's values have to lie together
        if t.stride() != (s * step, step, 1) and (_row_stride(name, t) or step) != step:
            raise ValueError(f"{name} has another token stride than the descriptor ({step})")
        ptrs.append(t.data_ptr())
    if h0 is None:
        ptrs.append(None)
    else:
        ptrs += _tensors_ok(dev, (("h0", h0, (b, w), torch.float32, True),))
    return dev, dt, ptrs


def _rec_forward(desc, x, g, z, h0, y, h_last, saved, want_saved, workspace):
    dev, dt, ins = _rec_inputs(desc, x, g, z, h0)
    shape, state = (desc.b, desc.s, desc.w), (desc.b, desc.w)
    if y is not None or h_last is not None:
        _tensors_ok(dev, (("y", y, shape, dt, True), ("h_last", h_last, state, torch.float32, True)))
    lib = _gpu(dev)
    ws = _buffer("workspace", moments_rec_workspace_size(desc, False), dev, workspace)
    if want_saved:
        saved = _buffer("saved", moments_rec_saved_size(desc), dev, saved)
    _wrote(y, h_last, saved)
    if y is None:
        y = _dense_like(x)
    if h_last is None:
        h_last = torch.empty(state, dtype=torch.float32, device=dev)
    head = (ctypes.byref(desc), *ins, y.data_ptr(), h_last.data_ptr())
    tail = _scratch(ws)
    if want_saved:
        _launch(dev, lib.moments_rec_fwd_save, *head, *_scratch(saved), *tail)
        return y, h_last, torch.empty(0, dtype=torch.uint8, device=dev) if saved is None else saved
    _launch(dev, lib.moments_rec_fwd, *head, *tail)
    return y, h_last


def moments_rec_fwd(desc: RecDesc, x, g, z=None, h0=None, y=None, h_last=None, workspace=None):
    """The gated recurrence over a whole sequence: returns (y [b,s,w] in the input dtype,
    h_last [b,w] float32)."""
    return _rec_forward(desc, x, g, z, h0, y, h_last, None, False, workspace)


def moments_rec_fwd_save(desc: RecDesc, x, g, z=None, h0=None, y=None, h_last=None, saved=None, workspace=None):
    """moments_rec_fwd that also keeps states along the sequences. Returns (y, h_last,
    saved); saved is opaque, for moments_rec_bwd_saved."""
    return _rec_forward(desc, x, g, z, h0, y, h_last, saved, True, workspace)


def moments_rec_bwd(desc: RecDesc, x, g, z, h0, d_y, d_h_last=None, want=("x", "g", "z", "h0"), out=None,
                    workspace=None, _saved=None):
    """Returns dict d_x, d_g, d_z (input dtype, dense), d_h0 (float32); None when not
    wanted (d_z, d_h0: or when there is no z, no h0)."""
    dev, dt, ins = _rec_inputs(desc, x, g, z, h0)
    cot = _tensors_ok(dev, (("d_y", d_y, (desc.b, desc.s, desc.w), dt, False),
                            ("d_h_last", d_h_last, (desc.b, desc.w), torch.float32, True)))
    out, grads = _gradients(dev, want, out, {"x": x, "g": g, "z": z, "h0": h0})
    lib = _lib.load()
    ws = _buffer("workspace", moments_rec_workspace_size(desc, True), dev, workspace)
    tail = (*cot, *grads, *_scratch(ws))
    if _saved is None:
        _launch(dev, lib.moments_rec_bwd, ctypes.byref(desc), *ins, *tail)
    else:
        sv = _buffer("saved", moments_rec_saved_size(desc), dev, _saved)
        _launch(dev, lib.moments_rec_bwd_saved, ctypes.byref(desc), *ins, *_scratch(sv), *tail)
    return out


def moments_rec_bwd_saved(desc: RecDesc, x, g, z, h0, saved, d_y, d_h_last=None, want=("x", "g", "z", "h0"),
                          out=None, workspace=None):
    """moments_rec_bwd reading what moments_rec_fwd_save kept. Same returns."""
    if saved is None:
        raise ValueError("saved is required")
    return moments_rec_bwd(desc, x, g, z, h0, d_y, d_h_last, want=want, out=out, workspace=workspace, _saved=saved)


def moments_rec_step(desc: RecDesc, x, g, z, state, slots=None, y=None):
    """One token of each sequence (s = 1) on a pool of states, state [nslots,w] float32,
    updated in place; ``slots`` as in moments_attn_step. Returns y [b,1,w]."""
    dev, dt, ins = _rec_inputs(desc, x, g, z, None)
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state must be a torch.Tensor [nslots,w]")
    n = state.shape[0]
    st, sl, out = _tensors_ok(dev, (("state", state, (n, desc.w), torch.float32, False),
                                    ("slots", slots, (desc.b,), torch.int32, True),
                                    ("y", y, (desc.b, desc.s, desc.w), dt, True)))
    lib = _gpu(dev)
    _wrote(state, y)
    if y is None:
        y = _dense_like(x)
        out = y.data_ptr()
    _launch(dev, lib.moments_rec_step, ctypes.byref(desc), *ins[:3], sl, n, st, out)
    return y


# ---------------------------------------------------------------- layer norm
def _flat_rows(name, t, w):
    """Rows of t [..., w] and the elements between them (0: dense)."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1 or t.shape[-1] != w:
        raise ValueError(f"{name} must be a torch.Tensor of rows of {w}")
    if t.is_contiguous() or t.numel() == 0:
        return (t.numel() // w if w else 0), 0
    n = t.numel() // w
    dims = [(size, step) for size, step in zip(t.shape[:-1], t.stride()[:-1]) if size > 1]
    step = dims[-1][1] if dims else w
    want = step
    for size, st in reversed(dims):
        if st != want:
            raise ValueError(f"{name} must have its rows a fixed stride apart")
        want = st * size
    if (w > 1 and t.stride(-1) != 1) or step < w:
        raise ValueError(f"{name} must hold each row's values together")
    return n, step if dims else 0


def ln_desc(x, eps=1e-5, residual=False) -> LnDesc:
    """Descriptor of layer norm for x [..., w], whose rows may be columns of a wider tensor
    (a fixed stride apart); ``residual``: with a float32 residual stream added before it."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a torch.Tensor of rows")
    n, step = _flat_rows("x", x, x.shape[-1])
    return LnDesc(n, x.shape[-1], step, BF16 if x.dtype is torch.bfloat16 else F32, int(bool(residual)), float(eps))


def moments_ln_workspace_size(desc: LnDesc) -> int:
    """Bytes of the backward's workspace (the forward needs none)."""
    return _size(_lib.load().moments_ln_workspace_size(ctypes.byref(desc)))


def _ln_x(desc, name, x, dt, stride):
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    n, step = _flat_rows(name, x, desc.w)
    if n != desc.n or x.dtype is not dt:
        raise ValueError(f"{name} must be {desc.n} rows of {dt}, got {n} of {x.dtype}")
    if n > 1 and (step or desc.w) != (stride or desc.w):
        raise ValueError(f"{name} has another row stride than the descriptor ({stride or desc.w})")
    return x.device


def moments_ln_fwd(desc: LnDesc, x, weight, bias=None, res=None, y=None, sum=None):
    """Returns (y, sum): the normed rows in the input dtype and, with a residual, x + res in
    float32 (else None), both of x's shape. ``sum`` may be ``res``."""
    dt = _DTYPES.get(desc.dtype)
    dev = _ln_x(desc, "x", x, dt, desc.x_stride)
    if not desc.residual and (res is not None or sum is not None):
        raise ValueError("res and sum must be None when the descriptor has no residual")
    f32 = torch.float32
    wp, bp, rp, yp, sp = _tensors_ok(dev, (
        ("weight", weight, (desc.w,), f32, False), ("bias", bias, (desc.w,), f32, True),
        ("res", res, x.shape, f32, not desc.residual), ("y", y, x.shape, dt, True), ("sum", sum, x.shape, f32, True)))
    lib = _gpu(dev)
    _wrote(y, sum)
    if y is None:
        y = _dense_like(x)
    if sum is None and desc.residual:
        sum = torch.empty_like(res)
    _launch(dev, lib.moments_ln_fwd, ctypes.byref(desc), x.data_ptr(), rp, wp, bp, y.data_ptr(),
            None if sum is None else sum.data_ptr())
    return y, sum


def moments_ln_bwd(desc: LnDesc, x, weight, bias, d_y, d_sum=None, want=("x", "res", "weight", "bias"), out=None,
                   workspace=None):
    """x is what was normed: the forward's sum with a residual, else its x. Returns dict
    d_x (input dtype, dense), d_res (float32, with a residual), d_weight, d_bias (float32);
    None when not wanted or not defined. d_res may be ``d_sum``."""
    dt, f32 = _DTYPES.get(desc.dtype), torch.float32
    dev = _ln_x(desc, "x", x, f32 if desc.residual else dt, 0 if desc.residual else desc.x_stride)
    if not desc.residual and d_sum is not None:
        raise ValueError("d_sum must be None when the descriptor has no residual")
    wp, _, yp, sp = _tensors_ok(dev, (("weight", weight, (desc.w,), f32, False), ("bias", bias, (desc.w,), f32, True),
                                      ("d_y", d_y, x.shape, dt, False), ("d_sum", d_sum, x.shape, f32, True)))
    like = {"x": _like(x.shape, dt), "res": _like(x.shape, f32) if desc.residual else None, "weight": weight,
            "bias": bias}
    out, grads = _gradients(dev, want, out, like)
    lib = _lib.load()
    ws = _buffer("workspace", moments_ln_workspace_size(desc), dev, workspace)
    _launch(dev, lib.moments_ln_bwd, ctypes.byref(desc), x.data_ptr(), wp, yp, sp, *grads, *_scratch(ws))
    return out


class _like:
    """Shape and dtype of a gradient, as _gradients reads them of an input."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype = shape, dtype


# ---------------------------------------------------------------- gradients' norm and clipping
class GradDesc:
    """Gradients and where their clipped values go; keeps the tensors. See grad_desc."""

    def __init__(self, grads, out):
        self.grads, self.in_place = list(grads), out is None
        self.out = list(self.grads if out is None else out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"out holds {len(self.out)} tensors, grads {len(self.grads)}")
        self.device = None
        spans = (_lib.Span * max(len(self.grads), 1))()
        for i, (t, o) in enumerate(zip(self.grads, self.out)):
            if not isinstance(t, torch.Tensor) or t.dtype not in (torch.float32, torch.bfloat16):
                raise ValueError(f"grads[{i}] must be a float32 or bfloat16 torch.Tensor")
            if self.device is None:
                self.device = t.device
            if t.device != self.device:
                raise ValueError(f"grads[{i}] is on {t.device}, the others on {self.device}")
            if not t.is_contiguous():
                raise ValueError(f"grads[{i}] must be contiguous")
            if o is not t:
                _expect(f"out[{i}]", o, t.shape, t.dtype, t.device)
            spans[i] = _lib.Span(t.data_ptr(), o.data_ptr(), t.numel(), BF16 if t.dtype is torch.bfloat16 else F32)
        self.spans, self.count = spans, len(self.grads)
        self._at = self._addresses()

    def _addresses(self):
        tensors = self.grads if self.in_place else self.grads + self.out
        return [*map(torch.Tensor.data_ptr, tensors)]


def grad_desc(grads, out=None) -> GradDesc:
    """Descriptor of many gradients (contiguous float32 or bfloat16 tensors on one device),
    for moments_grad_norm and moments_grad_clip; it keeps the tensors, which may be refilled
    between calls but not given other memory. It is of these tensors, not of the parameters:
    where a step gives the parameters new ones (``zero_grad()`` does, unless
    ``set_to_none=False``), each step makes its descriptor. ``out``: tensors like them that take
    the clipped values (None: in place). Raises if a tensor that is written overlaps another."""
    d = GradDesc(grads, out)
    rc = _lib.load().moments_grad_validate(d.spans, d.count)
    if rc == _lib.EINVAL:
        for name, tensors in (("grads", d.grads), ("out", d.out)):
            for i, t in enumerate(tensors):
                if t.data_ptr() % t.element_size():
                    raise ValueError(f"{name}[{i}] starts at {t.data_ptr():#x}, between two elements")
        raise ValueError("two of the tensors overlap (a gradient listed twice?)")
    _lib.check(rc)
    d.workspace_bytes = _size(_lib.load().moments_grad_workspace_size(d.spans, d.count))
    return d


def moments_grad_workspace_size(desc: GradDesc) -> int:
    return desc.workspace_bytes


def _grad_device(desc, norm):
    if desc._addresses() != desc._at:
        raise ValueError("a tensor of the descriptor has got other memory since (resize_, set_, .data): "
                         "make the descriptor again")
    dev = desc.device if desc.device is not None else (norm.device if isinstance(norm, torch.Tensor) else None)
    if dev is None:
        raise ValueError("norm is required when there are no gradients")
    return dev


def moments_grad_norm(desc: GradDesc, norm=None, workspace=None):
    """The root of the sum of all values' squares: a float32 scalar on the device. Ranks that
    hold shares of the gradients join their norms' squares before clipping."""
    dev = _grad_device(desc, norm)
    _tensors_ok(dev, (("norm", norm, (), torch.float32, True),))
    lib = _gpu(dev)
    ws = _buffer("workspace", desc.workspace_bytes, dev, workspace)
    _wrote(norm)
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=dev)
    _launch(dev, lib.moments_grad_norm, desc.spans, desc.count, norm.data_ptr(), *_scratch(ws))
    return norm


def moments_grad_clip(desc: GradDesc, norm, max_norm):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or into the
    descriptor's ``out``; a norm that is not finite leaves them as they are. Returns the
    tensors that hold the result."""
    dev = _grad_device(desc, norm)
    (at,) = _tensors_ok(dev, (("norm", norm, (), torch.float32, False),))
    lib = _gpu(dev)
    _wrote(*desc.out)
    _launch(dev, lib.moments_grad_clip, desc.spans, desc.count, at, float(max_norm))
    return desc.out


def kernel_chunk_len() -> int:
    """Tokens per kernel chunk (the kernels' own chunking, whatever chunk_len is)."""
    return int(_lib.load().moments_kernel_chunk_len())


def profile_enable(on: bool) -> bool:
    """Turn per-kernel HIP-event timing on or off; returns the previous state."""
    return bool(_lib.load().moments_profile_enable(int(bool(on))))


def profile_reset() -> None:
    _lib.load().moments_profile_reset()


def profile_read() -> dict:
    """{kernel name: (timed launches, summed ms)} of the launches timed so far."""
    lib = _lib.load()
    out = {}
    name = ctypes.c_char_p()
    n = ctypes.c_int64()
    ms = ctypes.c_double()
    count = lib.moments_profile_read(0, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms))
    _lib.check(min(count, 0))
    for i in range(count):
        lib.moments_profile_read(i, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms))
        out[name.value.decode()] = (int(n.value), float(ms.value))
    return out
