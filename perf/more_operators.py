"""The operators of a recurrent block's training and serving, as cases that can be timed and checked.

Three families:

* the gated linear recurrence over channels [b,s,w]: h[t] = a[t] h[t-1] + u[t], read as
  y[t] = h[t] silu(z[t]) (or y = h), with a decay for each channel and token. The gate g gives
  "log": a = exp(g), u = x; "mix": a = sigmoid(g), u = (1 - a) x; "unit": a = sigmoid(g),
  u = sqrt(1 - a^2) x. Whole sequences ("rec"), the same with gradients ("rec_train"), and one
  token for each sequence on a pool of states ("rec_step");
* layer norm of rows, with the residual stream added before it where there is one ("ln"), and
  the same with its gradients ("ln_train");
* the global norm of many gradients, and their clipping ("clip").

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is true, with this
package's entry points. ``exact`` gives the same results from the definitions in 64 bits: the
recurrence token by token with the derivatives of its single step, automatic differentiation of
the definition for the norm, sums in 64 bits for the gradients' norm.
"""
import math

import torch

own = False

GATES = ("log", "mix", "unit")
EPS = 1e-5        # of the layer norm
CLIP_EPS = 1e-6   # added to the gradients' norm


# ------------------------------------------------------------------------------------------------ the cases
def _rec(name, op, dtype, gate, b, s, w, **kw):
    case = dict(op=op, dtype=dtype, gate=gate, b=b, s=s, w=w, valid=s, ragged=False, resets=False, state=False,
                z=True, columns=False)
    case.update(kw)
    if name is not None:
        case["name"] = name
    return case


def _ln(name, op, dtype, n, w, **kw):
    case = dict(op=op, dtype=dtype, n=n, w=w, res=True, bias=True, offset=0.0)
    case.update(kw)
    if name is not None:
        case["name"] = name
    return case


def _clip(name, layers, width, inner, dtype, max_norm):
    case = dict(op="clip", layers=layers, width=width, inner=inner, dtype=dtype, max_norm=max_norm)
    if name is not None:
        case["name"] = name
    return case


def listed():
    return [
        # one short prompt of odd length: latency, and few chains to fill the card with
        _rec("rec_short_bf16", "rec", "bf16", "log", b=1, s=77, w=2048),
        # prompts of several lengths in one batch, each of packed documents (the state is cleared at each
        # document's first token), continued from cached states; inputs and gates are columns of one projection
        _rec("rec_packed_bf16", "rec", "bf16", "log", b=4, s=4096, w=2048, ragged=True, resets=True, state=True,
             columns=True),
        # the length and channels of the benchmark's long-context workload: few chains, each very long
        _rec("rec_long_s65536", "rec", "bf16", "unit", b=1, s=65536, w=4096, valid=60000),
        # odd sizes throughout, with an initial state and a cotangent of the last one (a sequence cut in pieces)
        _rec("rec_train_odd_f32", "rec_train", "f32", "unit", b=3, s=1533, w=509, ragged=True, state=True),
        # the sequences and channels of the benchmark's headline workload as a training step
        _rec("rec_train_bf16_b8_s8192", "rec_train", "bf16", "mix", b=8, s=8192, w=4096),
        # one token of one sequence: nothing but latency
        _rec("rec_step_one", "rec_step", "bf16", "mix", b=1, s=1, w=4096, pool=1),
        # one token for each sequence of a full batch, states scattered in a pool, some rows of the batch unused
        _rec("rec_step_batch256", "rec_step", "bf16", "log", b=256, s=1, w=4096, pool=300),
        # the rows of one decoding step: latency again
        _ln("ln_token_b32", "ln", "bf16", n=32, w=2048),
        # odd rows of a float32 model without a residual stream, values far from zero
        _ln("ln_train_odd_f32", "ln_train", "f32", n=4599, w=1021, res=False, offset=30.0),
        # the headline workload's tokens and channels as a training step
        _ln("ln_train_bf16_n65536", "ln_train", "bf16", n=65536, w=4096),
        # the few small parameters of one layer in float32, clipped
        _clip("clip_layer_f32", layers=1, width=128, inner=128, dtype="f32", max_norm=1.0),
        # several layers' bfloat16 matrices and float32 vectors, clipped
        _clip("clip_model_bf16", layers=7, width=4096, inner=4096, dtype="bf16", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rec", "rec", "rec_train", "rec_train", "rec_step", "ln", "ln_train", "clip"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "clip":
        width = _log(rng, 8, 2890)
        return _clip(None, layers=_log(rng, 1, 7), width=width, inner=rng.choice((width, 2 * width, width + 5)),
                     dtype=dtype, max_norm=rng.choice((0.1, 1.0, 1e9)))
    if op in ("ln", "ln_train"):
        n, w = _log(rng, 1, 65536), _log(rng, 16, 16384)
        if rng.random() < 0.6:
            w = max(8, w // 8 * 8)
        most = 1 << (26 if dtype == "f32" else 27)
        while n * w > most:
            n = (n + 1) // 2
        return _ln(None, op, dtype, n=n, w=w, res=rng.random() < 0.6, bias=rng.random() < 0.7,
                   offset=rng.choice((0.0, 0.0, 10.0)))
    gate, w = rng.choice(GATES), _log(rng, 1, 8192)
    if rng.random() < 0.6:
        w = max(8, w // 8 * 8)
    if op == "rec_step":
        b = _log(rng, 1, 256)
        return _rec(None, op, dtype, gate, b=b, s=1, w=min(w, 4096), z=rng.random() < 0.7,
                    pool=b + rng.choice((0, 1, 17)))
    b, s = _log(rng, 1, 8), _log(rng, 1, 32768)
    most = 1 << (25 if dtype == "f32" else 26)
    while b > 1 and b * s * w > most:
        b //= 2
    while s * w > most:
        s = (s + 1) // 2
    return _rec(None, op, dtype, gate, b=b, s=s, w=w, valid=s - rng.randrange(s // 8 + 1),
                ragged=rng.random() < 0.5, resets=rng.random() < 0.25, state=rng.random() < 0.5,
                z=rng.random() < 0.7, columns=rng.random() < 0.3)


# ------------------------------------------------------------------------------------------------ the inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    gen, dt = torch.Generator(device="cuda"), _dtype(case)
    gen.manual_seed(1_000_003 * int(seed) + 29)

    def randn(*shape, scale=1.0, to=dt):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(to)

    st = {"case": dict(case)}
    if case["op"] == "clip":
        return _prepare_clip(st, case, randn)
    if case["op"] in ("ln", "ln_train"):
        return _prepare_ln(st, case, randn)
    b, s, w = case["b"], case["s"], case["w"]
    # gates whose channels forget over one token up to some thousands, each token its own
    spread = torch.rand(w, device="cuda", generator=gen)
    noise = randn(b, s, w, to=torch.float32)
    if case["gate"] == "log":
        g = -torch.nn.functional.softplus(noise) * torch.exp(-8.0 * spread)
    else:
        g = noise + 8.0 * spread - 1.0
    del noise
    if case["resets"]:   # the first token of each packed document clears the state
        first = torch.rand(b, s, 1, device="cuda", generator=gen) < 1.0 / 200
        g = torch.where(first, torch.full_like(g, -math.inf), g)
    parts = {"x": randn(b, s, w), "g": g.to(dt), "z": randn(b, s, w) if case["z"] else None}
    del g
    if case["columns"]:  # one projection's output, cut
        names = [n for n in parts if parts[n] is not None]
        wide = torch.cat([parts[n] for n in names], -1)
        parts.update(zip(names, wide.split(w, dim=-1)))
    st.update(parts)
    if case["op"] == "rec_step":
        pool = case["pool"]
        st["state"] = randn(pool, w, scale=0.5, to=torch.float32)
        order = torch.randperm(pool, device="cuda", generator=gen)[:b].to(torch.int32)
        if b > 8:        # rows of the batch that hold no sequence at this step
            order[torch.randint(0, b, (b // 16,), device="cuda", generator=gen)] = -1
        st["slots"] = order
        return st
    st["lens"] = None
    if case["ragged"]:
        st["lens"] = torch.randint(0, s + 1, (b,), device="cuda", generator=gen).to(torch.int32)
        st["lens"][0] = s
    st["h0"] = randn(b, w, scale=0.5, to=torch.float32) if case["state"] else None
    if case["op"] == "rec_train":
        st["d_y"] = randn(b, s, w)
        st["d_h_last"] = randn(b, w, to=torch.float32) if case["state"] else None
    return st


def _prepare_ln(st, case, randn):
    n, w = case["n"], case["w"]
    st["x"] = (randn(n, w, to=torch.float32) + case["offset"]).to(_dtype(case))
    st["res"] = randn(n, w, scale=2.0, to=torch.float32) if case["res"] else None
    st["weight"] = 1.0 + randn(w, scale=0.1, to=torch.float32)
    st["bias"] = randn(w, scale=0.1, to=torch.float32) if case["bias"] else None
    if case["op"] == "ln_train":
        st["d_y"] = randn(n, w)
        st["d_sum"] = randn(n, w, to=torch.float32) if case["res"] else None
    return st


def _prepare_clip(st, case, randn):
    width, inner = case["width"], case["inner"]
    shapes = [(width, 2 * inner), (inner, width), (width, inner), (64, 128)]
    vectors = [(width,), (width,), (inner,), (2 * inner + 1,)]
    grads = []
    for _ in range(case["layers"]):
        grads += [randn(*s, scale=1e-2) for s in shapes] + [randn(*s, scale=1e-2, to=torch.float32) for s in vectors]
    st["grads"] = grads
    st["out"] = [torch.empty_like(g) for g in grads]   # the optimiser's own buffers
    if own:
        import mamba_ssm_chunkwise_amd as M
        st["desc"] = M.grad_desc(grads, out=st["out"])
    return st


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


# with this package -------------------------------------------------------------------------------
def _own_desc(st):
    import mamba_ssm_chunkwise_amd as M
    gate = {"log": M.GATE_LOG, "mix": M.GATE_MIX, "unit": M.GATE_UNIT}[st["case"]["gate"]]
    return M, M.rec_desc(st["x"], st["g"], st["z"], gate, valid_len=st["case"]["valid"], valid_lens=st.get("lens"))


def _own_rec(st):
    M, d = _own_desc(st)
    y, h_last = M.moments_rec_fwd(d, st["x"], st["g"], st["z"], st["h0"])
    return {"y": y, "h_last": h_last}


def _own_rec_train(st):
    M, d = _own_desc(st)
    x, g, z, h0 = st["x"], st["g"], st["z"], st["h0"]
    y, h_last, saved = M.moments_rec_fwd_save(d, x, g, z, h0)
    out = M.moments_rec_bwd_saved(d, x, g, z, h0, saved, st["d_y"], st["d_h_last"])
    out["y"] = y
    out["h_last"] = h_last
    return out


def _own_rec_step(st):
    M, d = _own_desc(st)
    y = M.moments_rec_step(d, st["x"], st["g"], st["z"], st["state"], st["slots"])
    return {"y": y, "state": st["state"]}


def _own_ln(st):
    import mamba_ssm_chunkwise_amd as M
    d = M.ln_desc(st["x"], eps=EPS, residual=st["res"] is not None)
    y, total = M.moments_ln_fwd(d, st["x"], st["weight"], st["bias"], st["res"])
    return {"y": y, "sum": total}


def _own_ln_train(st):
    import mamba_ssm_chunkwise_amd as M
    d = M.ln_desc(st["x"], eps=EPS, residual=st["res"] is not None)
    y, total = M.moments_ln_fwd(d, st["x"], st["weight"], st["bias"], st["res"])
    out = M.moments_ln_bwd(d, st["x"] if total is None else total, st["weight"], st["bias"], st["d_y"], st["d_sum"])
    out.update(y=y, sum=total)
    return out


def _own_clip(st):
    import mamba_ssm_chunkwise_amd as M
    norm = M.moments_grad_norm(st["desc"])
    M.moments_grad_clip(st["desc"], norm, st["case"]["max_norm"])
    return [norm, *st["out"]]


_OWN = {"rec": _own_rec, "rec_train": _own_rec_train, "rec_step": _own_rec_step, "ln": _own_ln,
        "ln_train": _own_ln_train, "clip": _own_clip}


# in plain torch ----------------------------------------------------------------------------------
def _lens(st):
    """Valid tokens of each sequence, [b]."""
    case = st["case"]
    top = min(case["valid"], case["s"])
    if st.get("lens") is None:
        return torch.full((case["b"],), top, device="cuda")
    return st["lens"].clamp(0, top).long()


def _gates(g, x, gate):
    """The decay a, 1 - a, the input's factor and the input as it enters the state, in float32."""
    if gate == "log":
        return torch.exp(g), None, None, x
    a, b = torch.sigmoid(g), torch.sigmoid(-g)
    f = b if gate == "mix" else torch.sqrt(b * (1.0 + a))
    return a, b, f, f * x


def _scan(a, u, first):
    """h[t] = a[t] h[t-1] + u[t] over dim 1 from h[-1] = first: every chunk from zero with the product of its
    decays, the chunks' ends one after the other, then what enters each chunk added to it."""
    b, s, w = a.shape
    n = 1 << max(0, (max(s, 1) - 1).bit_length() + 1 >> 1)       # tokens of a chunk, about the root of s
    nc = -(-s // n)
    pad = nc * n - s
    A = torch.nn.functional.pad(a, (0, 0, 0, pad), value=1.0).reshape(b, nc, n, w)
    H = torch.nn.functional.pad(u, (0, 0, 0, pad)).reshape(b, nc, n, w)
    A, H = (A.clone(), H.clone()) if pad == 0 else (A, H)
    for t in range(1, n):
        H[:, :, t] += A[:, :, t] * H[:, :, t - 1]
        A[:, :, t] *= A[:, :, t - 1]
    into = torch.empty(b, nc, w, device=a.device)
    at = first
    for c in range(nc):
        into[:, c] = at
        at = torch.addcmul(H[:, c, -1], A[:, c, -1], at)
    return torch.addcmul(H, A, into[:, :, None]).reshape(b, nc * n, w)[:, :s]


def _plain_fwd(st):
    case = st["case"]
    live = (torch.arange(case["s"], device="cuda")[None, :] < _lens(st)[:, None])[:, :, None]
    x = torch.where(live, st["x"].float(), 0.0)
    g = torch.where(live, st["g"].float(), 0.0)
    a, b, f, u = _gates(g, x, case["gate"])
    a, u = torch.where(live, a, 1.0), torch.where(live, u, 0.0)     # padding hands the state on
    first = st["h0"] if st["h0"] is not None else torch.zeros(case["b"], case["w"], device="cuda")
    h = _scan(a, u, first)
    y = h
    sig = None
    if st["z"] is not None:
        z = torch.where(live, st["z"].float(), 0.0)
        sig = torch.sigmoid(z)
        y = h * (z * sig)
    y = torch.where(live, y, 0.0).to(st["x"].dtype)
    return dict(live=live, x=x, a=a, b=b, f=f, first=first, h=h, sig=sig, y=y, last=h[:, -1])


def _plain_rec(st):
    f = _plain_fwd(st)
    return {"y": f["y"], "h_last": f["last"].contiguous()}


def _plain_rec_train(st):
    case, dt = st["case"], st["x"].dtype
    p = _plain_fwd(st)
    live, x, a, h, sig = (p[n] for n in ("live", "x", "a", "h", "sig"))
    dy = torch.where(live, st["d_y"].float(), 0.0)
    d_z, src = None, dy
    if sig is not None:
        z = torch.where(live, st["z"].float(), 0.0)
        d_z = (dy * h * (sig * (1.0 + z * (1.0 - sig)))).to(dt)
        src = dy * (z * sig)
    d_last = st["d_h_last"] if st["d_h_last"] is not None else torch.zeros_like(p["first"])
    # the state's cotangent, from the last token to the first: token t's decay is applied after it
    nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    delta = _scan(nxt.flip(1), src.flip(1), d_last).flip(1)
    before = torch.cat([p["first"][:, None], h[:, :-1]], 1)
    if case["gate"] == "log":
        d_x, d_g = delta, a * before * delta
    else:
        b, f = p["b"], p["f"]
        own_part = x if case["gate"] == "mix" else (a / (1.0 + a)) * (f / b.clamp(min=1e-38)) * x
        d_x = f * delta
        d_g = a * b * (before - own_part) * delta
    d_x, d_g = (torch.where(live, t, 0.0).to(dt) for t in (d_x, d_g))
    return {"y": p["y"], "h_last": p["last"].contiguous(), "d_x": d_x, "d_g": d_g, "d_z": d_z,
            "d_h0": a[:, 0] * delta[:, 0] if st["h0"] is not None else None}


def _plain_rec_step(st):
    case, state = st["case"], st["state"]
    used = st["slots"] >= 0
    at = st["slots"].clamp(min=0).long()
    a, _, _, u = _gates(st["g"][:, 0].float(), st["x"][:, 0].float(), case["gate"])
    old = state[at]
    new = torch.addcmul(u, a, old)
    y = new
    if st["z"] is not None:
        z = st["z"][:, 0].float()
        y = new * (z * torch.sigmoid(z))
    # each slot's row of the batch, -1 for none; rows without a sequence write past the pool's end
    row = torch.full((state.shape[0] + 1,), -1, device="cuda")
    row[torch.where(used, at, state.shape[0])] = torch.arange(case["b"], device="cuda")
    row = row[:-1]
    state.copy_(torch.where((row >= 0)[:, None], new[row.clamp(min=0)], state))
    return {"y": torch.where(used[:, None], y, 0.0)[:, None].to(st["x"].dtype), "state": state}


def _plain_norm(st):
    s = st["x"].float()
    if st["res"] is not None:
        s = s + st["res"]
    d = s - s.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)
    xhat = d * rstd
    y = xhat * st["weight"]
    if st["bias"] is not None:
        y = y + st["bias"]
    return s, xhat, rstd, y.to(st["x"].dtype)


def _plain_ln(st):
    s, _, _, y = _plain_norm(st)
    return {"y": y, "sum": s if st["res"] is not None else None}


def _plain_ln_train(st):
    dt, res = st["x"].dtype, st["res"] is not None
    s, xhat, rstd, y = _plain_norm(st)
    dy = st["d_y"].float()
    gy = dy * st["weight"]
    d = (gy - gy.mean(-1, keepdim=True) - xhat * (gy * xhat).mean(-1, keepdim=True)) * rstd
    if res:
        d = d + st["d_sum"]
    return {"y": y, "sum": s if res else None, "d_x": d.to(dt), "d_res": d if res else None,
            "d_weight": (dy * xhat).sum(0), "d_bias": dy.sum(0) if st["bias"] is not None else None}


def _plain_clip(st):
    norm = torch.sqrt(torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum()).float()
    factor = torch.clamp(st["case"]["max_norm"] / (norm + CLIP_EPS), max=1.0)
    for g, o in zip(st["grads"], st["out"]):
        o.copy_(g.float() * factor)
    return [norm, *st["out"]]


_PLAIN = {"rec": _plain_rec, "rec_train": _plain_rec_train, "rec_step": _plain_rec_step, "ln": _plain_ln,
          "ln_train": _plain_ln_train, "clip": _plain_clip}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        return _exact_clip(st)
    if case["op"] in ("ln", "ln_train"):
        return _exact_ln(st)
    if case["op"] == "rec_step":
        return _exact_step(st)
    return _exact_rec(st)


def _one_step(gate, x, g, before):
    """The recurrence's single step, as it is defined."""
    if gate == "log":
        return torch.exp(g) * before + x
    a, rest = torch.sigmoid(g), torch.sigmoid(-g)
    if gate == "mix":
        return a * before + rest * x
    return a * before + torch.sqrt(rest + rest * a) * x


def _read(h, z):
    return h if z is None else h * z / (1.0 + torch.exp(-z))


def _exact_step(st):
    case = st["case"]
    state = st["state"].double()
    y = torch.zeros(case["b"], 1, case["w"], dtype=torch.float64, device="cuda")
    for i, slot in enumerate(st["slots"].tolist()):
        if slot < 0:
            continue
        state[slot] = _one_step(case["gate"], st["x"][i, 0].double(), st["g"][i, 0].double(), state[slot])
        y[i, 0] = _read(state[slot], None if st["z"] is None else st["z"][i, 0].double())
    return {"y": y, "state": state}


def _exact_rec(st):
    """One sequence at a time, token by token: the state forwards, its cotangent backwards."""
    case = st["case"]
    b, s, w, gate = (case[k] for k in ("b", "s", "w", "gate"))
    train = case["op"] == "rec_train"
    if b * s * (2 if train else 1) > 600_000:
        return None      # over 20 seconds of single tokens
    names = ["y", "d_x", "d_g", "d_z"] if train else ["y"]
    out = {n: torch.zeros(b, s, w, dtype=torch.float64, device="cuda") for n in names if n != "d_z" or case["z"]}
    out["h_last"] = torch.zeros(b, w, dtype=torch.float64, device="cuda")
    if train:
        out["d_z"] = out.get("d_z")
        out["d_h0"] = torch.zeros_like(out["h_last"]) if st["h0"] is not None else None
    for i, n in enumerate(_lens(st).tolist()):
        x, g = st["x"][i, :n].double(), st["g"][i, :n].double()
        z = st["z"][i, :n].double() if case["z"] else None
        a = torch.exp(g) if gate == "log" else torch.sigmoid(g)
        states = torch.empty(n + 1, w, dtype=torch.float64, device="cuda")
        states[0] = st["h0"][i].double() if st["h0"] is not None else 0.0
        u = _one_step(gate, x, g, torch.zeros_like(x))
        for t in range(n):
            torch.addcmul(u[t], a[t], states[t], out=states[t + 1])
        del u
        out["h_last"][i] = states[n]
        out["y"][i, :n] = _read(states[1:], z)
        if not train:
            continue
        dy = st["d_y"][i, :n].double()
        delta = dy if z is None else _read(dy, z)
        delta = delta.clone()
        if n > 0:
            if st["d_h_last"] is not None:
                delta[n - 1] += st["d_h_last"][i].double()
            for t in range(n - 1, 0, -1):
                delta[t - 1].addcmul_(a[t], delta[t])
            if st["h0"] is not None:
                out["d_h0"][i] = a[0] * delta[0]
            with torch.enable_grad():
                leaf = [x.requires_grad_(), g.requires_grad_()]
                out["d_x"][i, :n], out["d_g"][i, :n] = torch.autograd.grad(
                    _one_step(gate, x, g, states[:-1]), leaf, delta)
                if z is not None:
                    out["d_z"][i, :n] = torch.autograd.grad(_read(states[1:], z.requires_grad_()), z, dy)[0]
        elif st["h0"] is not None:
            out["d_h0"][i] = st["d_h_last"][i].double()
    return out


def _exact_ln(st):
    """Automatic differentiation of the definition, some rows at a time."""
    train, res = st["case"]["op"] == "ln_train", st["res"] is not None
    n, w = st["x"].shape
    weight = st["weight"].double().requires_grad_(train)
    bias = st["bias"].double().requires_grad_(train) if st["bias"] is not None else None
    out = {"y": torch.empty(n, w, dtype=torch.float64, device="cuda"), "sum": None}
    if res:
        out["sum"] = st["x"].double() + st["res"].double()
    if train:
        d = torch.empty(n, w, dtype=torch.float64, device="cuda")
        d_weight = torch.zeros(w, dtype=torch.float64, device="cuda")
        d_bias = torch.zeros_like(d_weight)
    step = max(1, (1 << 25) // w)
    for i in range(0, n, step):
        s = (out["sum"] if res else st["x"])[i:i + step].double().requires_grad_(train)
        c = s - s.sum(-1, keepdim=True) / w
        y = c / torch.sqrt((c ** 2).sum(-1, keepdim=True) / w + EPS) * weight
        if bias is not None:
            y = y + bias
        out["y"][i:i + step] = y.detach()
        if train:
            leaves = [s, weight] + ([bias] if bias is not None else [])
            got = torch.autograd.grad(y, leaves, st["d_y"][i:i + step].double())
            d[i:i + step] = got[0]
            d_weight += got[1]
            if bias is not None:
                d_bias += got[2]
    if train:
        if res:
            d += st["d_sum"]
        out.update(d_x=d, d_res=d if res else None, d_weight=d_weight, d_bias=d_bias if bias is not None else None)
    return out


def _exact_clip(st):
    total = 0.0
    for g in st["grads"]:
        total += float(torch.linalg.vector_norm(g.double()) ** 2)
    norm = math.sqrt(total)
    factor = min(1.0, st["case"]["max_norm"] / (norm + CLIP_EPS))
    return [torch.tensor(norm, dtype=torch.float64, device="cuda"), *[g.double() * factor for g in st["grads"]]]


# ------------------------------------------------------------------------------------------------ what it takes
def work(case):
    """Bytes of every input once and every output once; operations of each element."""
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "clip":
        width, inner = case["width"], case["inner"]
        mats = case["layers"] * (4 * width * inner + 64 * 128)
        vecs = case["layers"] * (2 * width + 3 * inner + 1)
        return {"bytes": 2 * (e * mats + 4 * vecs) + 4, "flops": 3 * (mats + vecs)}
    if case["op"] in ("ln", "ln_train"):
        n, w = case["n"], case["w"]
        params = 4 * w * (2 if case["bias"] else 1)
        fwd = n * w * (2 * e + (8 if case["res"] else 0)) + params
        if case["op"] == "ln":
            return {"bytes": fwd, "flops": 8 * n * w}
        return {"bytes": fwd + n * w * (2 * e + (8 if case["res"] else 0)) + params, "flops": 24 * n * w}
    b, s, w = case["b"], case["s"], case["w"]
    nin = 3 if case["z"] else 2
    if case["op"] == "rec_step":
        return {"bytes": b * (w * (8 + e * (nin + 1)) + 4), "flops": 10 * b * w}
    rows = b * min(case["valid"], s) // (2 if case["ragged"] else 1)     # ragged lengths: half on average
    states = 4 * b * w * (2 if case["state"] else 1)
    if case["op"] == "rec":
        return {"bytes": e * w * (nin * rows + b * s) + states, "flops": 10 * rows * w}
    return {"bytes": e * w * ((nin + 1) * rows + (1 + nin) * b * s) + states + (8 * b * w if case["state"] else 0),
            "flops": 30 * rows * w}
