"""The operators around the state scan, as cases that can be timed and checked.

Two families, in the layouts of the state-moments path (xhat [b,s,c,h,p], bhat
[b,s,c,g,r], da [b,s,h]; c channels share a token, g groups of heads share a key):

* linear attention with a decay for each head: y[t] = qhat[t] . h~[t] over the
  states h~[t] = exp(da[t]) h~[t-1] + sum_c xhat[t,c] (outer) bhat[t,c]; the
  chunked form for prompts ("prefill"), the same with its gradients ("train"),
  and one token per sequence on a pool of states ("step");
* norms of queries and keys for each head with the position rotation in the same
  pass ("qk"), and the same with its gradients ("qk_train").

``run`` computes a case in plain torch operations in 32 bits, or, where ``own``
is true, with this package's entry points. ``exact`` gives the same results from
the definitions in 64 bits: the recurrence token by token for the attention,
automatic differentiation of the definition for the norms.
"""
import math

import torch

own = False

ROTS = ("none", "pairwise", "half", "quat")
CHUNK = 64      # tokens per chunk of the plain chunked form
RESET = -110.0  # log-decays below this are a decay of exactly zero in 32 bits
EPS = 1e-5      # of the norms


# ------------------------------------------------------------------------------------------------ the cases
def _attn(name, op, dtype, b, s, c, h, g, p, r, **kw):
    case = dict(op=op, dtype=dtype, b=b, s=s, c=c, h=h, g=g, p=p, r=r, valid=s, ragged=False, resets=False,
                state=False)
    case.update(kw)
    if name is not None:
        case["name"] = name
    return case


def _qk(name, op, dtype, b, s, c, h, g, r, rot, width, **kw):
    case = dict(op=op, dtype=dtype, b=b, s=s, c=c, h=h, g=g, r=r, rot=rot, width=width, rot_h=h, bias=True,
                stride=0)
    case.update(kw)
    if name is not None:
        case["name"] = name
    return case


def listed():
    return [
        # one short prompt of odd length: latency, and few chains to fill the card with
        _attn("prefill_short_bf16", "prefill", "bf16", b=1, s=77, c=1, h=32, g=32, p=64, r=128),
        # the float32 half-split workload of the benchmark, its padded tail included
        _attn("prefill_f32_b2_s2048", "prefill", "f32", b=2, s=2048, c=2, h=16, g=16, p=64, r=64, valid=1900),
        # prompts of several lengths in one batch, each of packed documents (the state is cleared at each
        # document's first token), continued from cached states, keys shared by groups of four heads
        _attn("prefill_packed_bf16", "prefill", "bf16", b=4, s=4096, c=1, h=32, g=8, p=64, r=128, ragged=True,
              resets=True, state=True),
        # the long-context workload of the benchmark: few chains, each very long
        _attn("prefill_long_s65536", "prefill", "bf16", b=1, s=65536, c=4, h=32, g=32, p=128, r=128, valid=60000),
        # odd sizes throughout, with an initial state and a cotangent of the last one (a sequence cut in pieces)
        _attn("train_odd_f32", "train", "f32", b=3, s=509, c=3, h=6, g=2, p=37, r=45, ragged=True, state=True),
        # the benchmark's mid-size bfloat16 workload as a training step
        _attn("train_bf16_b4_s4096", "train", "bf16", b=4, s=4096, c=1, h=32, g=32, p=64, r=128),
        # the benchmark's headline workload as a training step
        _attn("train_bf16_b8_s8192", "train", "bf16", b=8, s=8192, c=2, h=64, g=64, p=64, r=128),
        # one token of one sequence: nothing but latency
        _attn("step_one", "step", "bf16", b=1, s=1, c=2, h=64, g=64, p=64, r=128, valid=1, pool=1),
        # one token for each sequence of a full batch, states scattered in a pool, some rows of the batch unused
        _attn("step_batch256", "step", "bf16", b=256, s=1, c=1, h=64, g=8, p=64, r=128, valid=1, pool=300),
        # the queries and keys of one decoding step, cut out of a wider projection
        _qk("qk_token_b32", "qk", "bf16", b=32, s=1, c=1, h=32, g=8, r=128, rot="quat", width=8, stride=6144),
        # the float32 half-split workload with gradients; one rotation for all heads
        _qk("qk_train_f32", "qk_train", "f32", b=2, s=2048, c=2, h=16, g=16, r=64, rot="half", width=16, rot_h=1),
        # the headline workload with gradients; keys and queries projected for eight groups of heads
        _qk("qk_train_bf16_b8_s8192", "qk_train", "bf16", b=8, s=8192, c=2, h=64, g=8, r=128, rot="pairwise",
            width=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "train", "train", "step", "qk", "qk_train"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    c = rng.choice((1, 1, 2, 3, 4))
    g = rng.choice((1, 2, 4, 8, 16, 32))
    h = g * rng.choice((1, 1, 2, 4))
    r = rng.choice((16, 24, 45, 64, 96, 128, 128))
    p = rng.choice((16, 37, 64, 64, 96, 128))
    if op == "step":
        b = _log(rng, 1, 256)
        return _attn(None, op, dtype, b=b, s=1, c=c, h=min(h, 64), g=min(g, h), p=p, r=r, valid=1,
                     pool=b + rng.choice((0, 1, 17)))
    s = _log(rng, 1, 16384)
    b = _log(rng, 1, 8)
    while b > 1 and b * s * c * h > (1 << 21):
        b //= 2
    while s * c * h > (1 << 21):
        s = (s + 1) // 2
    if op in ("prefill", "train"):
        return _attn(None, op, dtype, b=b, s=s, c=c, h=h, g=g, p=p, r=r, valid=s - rng.randrange(s // 8 + 1),
                     ragged=rng.random() < 0.5, resets=rng.random() < 0.25, state=rng.random() < 0.5)
    rot = rng.choice(ROTS)
    if rot == "half" and r % 2:
        rot = "pairwise"
    full = r // 4 if rot == "quat" else r // 2
    width = 0 if rot == "none" else rng.choice((full, max(1, full // 2), max(1, full // 3)))
    row = c * g * r
    return _qk(None, op, dtype, b=b, s=s, c=c, h=h, g=g, r=r, rot=rot, width=width,
               rot_h=rng.choice((h, h, 1)), bias=rng.random() < 0.7, stride=rng.choice((0, row + 8, 2 * row)))


# ------------------------------------------------------------------------------------------------ the inputs
def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * int(seed) + 17)
    return g


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    gen, dt = _gen(case, seed), _dtype(case)

    def randn(*shape, scale=1.0, to=dt):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(to)

    b, s, c, h, g, r = (case[k] for k in ("b", "s", "c", "h", "g", "r"))
    st = {"case": dict(case)}
    if case["op"] in ("qk", "qk_train"):
        row, stride = c * g * r, case["stride"]
        for name in ("q", "k"):
            if stride:   # columns of a wider projection
                st[name] = randn(b, s, stride)[:, :, :row].view(b, s, c, g, r)
            else:
                st[name] = randn(b, s, c, g, r)
            st["w" + name] = 1.0 + randn(r, scale=0.1, to=torch.float32)
            st["b" + name] = randn(h, r, scale=0.1, to=torch.float32) if case["bias"] else None
        st["rot"] = None
        if case["rot"] == "quat":
            v = randn(b, s, case["rot_h"], case["width"], 4, to=torch.float32)
            st["rot"] = (v / v.norm(dim=-1, keepdim=True)).to(dt)
        elif case["rot"] != "none":
            inc = randn(b, s, case["rot_h"], case["width"], scale=0.05, to=torch.float32)
            st["rot"] = torch.cumsum(inc, dim=1).to(dt)
        if case["op"] == "qk_train":
            st["d_qhat"], st["d_khat"] = randn(b, s, c, h, r), randn(b, s, c, h, r)
        return st
    p = case["p"]
    st["xhat"] = randn(b, s, c, h, p)
    st["bhat"] = randn(b, s, c, g, r)
    st["qhat"] = randn(b, s, c, g, r, scale=r ** -0.5)
    da = -torch.nn.functional.softplus(randn(b, s, h, to=torch.float32) - 1.0)
    if case["resets"]:   # the first token of each packed document clears the state
        first = torch.rand(b, s, 1, device="cuda", generator=gen) < 1.0 / 200
        da = torch.where(first, torch.full_like(da, -math.inf), da)
    st["da"] = da.to(dt)
    if case["op"] == "step":
        pool = case["pool"]
        st["state"] = randn(pool, h, p, r, scale=0.5, to=torch.float32)
        order = torch.randperm(pool, device="cuda", generator=gen)[:b].to(torch.int32)
        if b > 8:        # rows of the batch that hold no sequence at this step
            order[torch.randint(0, b, (b // 16,), device="cuda", generator=gen)] = -1
        st["slots"] = order
        return st
    st["lens"] = None
    if case["ragged"]:
        st["lens"] = torch.randint(0, s + 1, (b,), device="cuda", generator=gen).to(torch.int32)
        st["lens"][0] = s
    st["h0"] = randn(b, h, p, r, scale=0.5, to=torch.float32) if case["state"] else None
    if case["op"] == "train":
        st["d_y"] = randn(b, s, c, h, p)
        st["d_h_last"] = randn(b, h, p, r, scale=0.1, to=torch.float32) if case["state"] else None
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
    return M, M.attn_desc(st["xhat"], st["bhat"], valid_len=st["case"]["valid"], valid_lens=st.get("lens"))


def _own_prefill(st):
    M, d = _own_desc(st)
    y, h_last = M.moments_attn_fwd(d, st["xhat"], st["bhat"], st["qhat"], st["da"], st["h0"])
    return {"y": y, "h_last": h_last}


def _own_train(st):
    M, d = _own_desc(st)
    x, k, q, da, h0 = st["xhat"], st["bhat"], st["qhat"], st["da"], st["h0"]
    y, h_last, saved = M.moments_attn_fwd_save(d, x, k, q, da, h0)
    out = M.moments_attn_bwd_saved(d, x, k, q, da, h0, saved, st["d_y"], st["d_h_last"])
    out["y"] = y
    if h0 is not None:
        out["h_last"] = h_last
    return out


def _own_step(st):
    M, d = _own_desc(st)
    y = M.moments_attn_step(d, st["xhat"], st["bhat"], st["qhat"], st["da"], st["state"], st["slots"])
    return {"y": y, "state": st["state"]}


def _own_qk_desc(st):
    import mamba_ssm_chunkwise_amd as M
    case = st["case"]
    kind = {"none": M.ROT_NONE, "pairwise": M.ROT_PAIRWISE, "half": M.ROT_HALF, "quat": M.ROT_QUAT}[case["rot"]]
    return M, M.qk_desc(st["q"], st["k"], case["h"], kind, rot=st["rot"], eps=EPS)


def _own_qk(st):
    M, d = _own_qk_desc(st)
    qhat, khat = M.moments_qk_fwd(d, st["q"], st["k"], st["wq"], st["wk"], st["bq"], st["bk"], st["rot"])
    return {"qhat": qhat, "khat": khat}


def _own_qk_train(st):
    M, d = _own_qk_desc(st)
    args = (st["q"], st["k"], st["wq"], st["wk"], st["bq"], st["bk"], st["rot"])
    qhat, khat = M.moments_qk_fwd(d, *args)
    out = M.moments_qk_bwd(d, *args, st["d_qhat"], st["d_khat"])
    out.update(qhat=qhat, khat=khat)
    return out


_OWN = {"prefill": _own_prefill, "train": _own_train, "step": _own_step, "qk": _own_qk, "qk_train": _own_qk_train}


# in plain torch ----------------------------------------------------------------------------------
def _lens(st):
    """Valid tokens of each sequence, [b]."""
    case = st["case"]
    top = min(case["valid"], case["s"])
    if st.get("lens") is None:
        return torch.full((case["b"],), top, device="cuda")
    return st["lens"].clamp(0, top).long()


def _rows(x, case, nc, live):
    """[b,s,c,n,w] -> [b,h,chunks,CHUNK*c,w] in float32 for every head, zero where a token is padding."""
    b, s, c, n, w = x.shape
    x = torch.where(live[:, :, None, None, None], x.float(), 0.0)
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 0, 0, nc * CHUNK - s))
    x = x.permute(0, 3, 1, 2, 4).reshape(b, n, nc, CHUNK * c, w)
    return x if n == case["h"] else x.repeat_interleave(case["h"] // n, dim=1)


def _unrows(x, case, heads, dt):
    """[b,h,chunks,CHUNK*c,w] -> [b,s,c,heads,w], summed over the heads of a group, rounded once."""
    b, s, c, h = case["b"], case["s"], case["c"], case["h"]
    w = x.shape[-1]
    x = x.reshape(b, h, -1, c, w)[:, :, :s]
    if heads != h:
        x = x.reshape(b, heads, h // heads, s, c, w).sum(2)
    return x.permute(0, 2, 3, 1, 4).to(dt).contiguous()


def _segsum(a):
    """out[.., t, j] = sum of a[.., i] over j < i <= t, -inf above the diagonal; no difference of long sums."""
    n = a.shape[-1]
    i = torch.arange(n, device=a.device)
    x = torch.where(i[:, None] > i[None, :], a[..., :, None], 0.0).cumsum(-2)
    return torch.where(i[:, None] >= i[None, :], x, -math.inf)


def _decays(st, nc, live):
    """Per chunk: L over rows, the decay from the chunk's start to each row, from each row to its end, and over
    the whole chunk."""
    case = st["case"]
    c = case["c"]
    a = torch.where(live[:, :, None], st["da"].float().clamp(min=RESET), 0.0)
    a = torch.nn.functional.pad(a, (0, 0, 0, nc * CHUNK - case["s"])).permute(0, 2, 1)
    a = a.reshape(a.shape[0], a.shape[1], nc, CHUNK)
    L = torch.exp(_segsum(a)).repeat_interleave(c, -1).repeat_interleave(c, -2)
    start = torch.exp(a.cumsum(-1)).repeat_interleave(c, -1)[..., None]
    end = torch.exp(a.flip(-1).cumsum(-1).flip(-1) - a).repeat_interleave(c, -1)[..., None]
    return a, L, start, end


def _carry(local, total, first, back=False):
    """The state before each chunk (after it, with ``back``) and past the last one, from the chunks' own sums."""
    if back:
        local, total = local.flip(2), total.flip(2)
    zero = torch.zeros_like(total[..., :1])
    D = torch.exp(_segsum(torch.cat([zero, total], -1)))          # from the point i to the point n, i <= n
    src = torch.cat([first[:, :, None], local], 2)
    b, h, n = src.shape[:3]
    pts = torch.matmul(D.reshape(b * h, n, n), src.reshape(b * h, n, -1)).reshape(src.shape)
    into, last = pts[:, :, :-1], pts[:, :, -1]
    return (into.flip(2) if back else into), last


def _plain_fwd(st):
    case = st["case"]
    nc = max(1, -(-case["s"] // CHUNK))
    live = torch.arange(case["s"], device="cuda")[None, :] < _lens(st)[:, None]
    x, k, q = (_rows(st[n], case, nc, live) for n in ("xhat", "bhat", "qhat"))
    a, L, start, end = _decays(st, nc, live)
    S = torch.matmul(q, k.transpose(-1, -2).contiguous()) * L
    first = st["h0"].float() if st["h0"] is not None else torch.zeros(
        case["b"], case["h"], case["p"], case["r"], device="cuda")
    H, last = _carry(torch.matmul((x * end).transpose(-1, -2).contiguous(), k), a.sum(-1), first)
    y = torch.matmul(S, x) + torch.matmul(q, H.transpose(-1, -2).contiguous()) * start
    return dict(nc=nc, live=live, x=x, k=k, q=q, a=a, L=L, start=start, end=end, S=S, H=H, y=y, last=last)


def _plain_prefill(st):
    f = _plain_fwd(st)
    return {"y": _unrows(f["y"], st["case"], st["case"]["h"], st["xhat"].dtype), "h_last": f["last"]}


def _plain_train(st):
    case, dt = st["case"], st["xhat"].dtype
    f = _plain_fwd(st)
    x, k, q, a, L, start, end, H = (f[n] for n in ("x", "k", "q", "a", "L", "start", "end", "H"))
    b, h, c, g, s, nc = case["b"], case["h"], case["c"], case["g"], case["s"], f["nc"]
    dy = _rows(st["d_y"], case, nc, f["live"])
    T = torch.matmul(dy, x.transpose(-1, -2).contiguous()) * L
    d_last = st["d_h_last"].float() if st["d_h_last"] is not None else torch.zeros_like(f["last"])
    local = torch.matmul((dy * start).transpose(-1, -2).contiguous(), q)
    G, d_h0 = _carry(local, a.sum(-1), d_last, back=True)     # cotangent of the state after each chunk
    q_in = torch.matmul(dy, H) * start
    k_in = torch.matmul(x, G) * end
    d_q = torch.matmul(T, k) + q_in
    d_k = torch.matmul(T.transpose(-1, -2).contiguous(), q) + k_in
    d_x = torch.matmul(f["S"].transpose(-1, -2).contiguous(), dy) + torch.matmul(
        k, G.transpose(-1, -2).contiguous()) * end
    # the log-decay of a token scales whatever crosses it: pairs inside the chunk, the entering state as read
    # from it on, the writes before it as the rest of the sequence reads them, and the state passing through
    u = (q * q_in).sum(-1).reshape(b, h, nc, CHUNK, c).sum(-1)
    v = (k * k_in).sum(-1).reshape(b, h, nc, CHUNK, c).sum(-1)
    A = (torch.matmul(q, k.transpose(-1, -2).contiguous()) * T).reshape(b, h, nc, CHUNK, c, CHUNK, c).sum((4, 6))
    below = A.flip(-2).cumsum(-2).flip(-2)                    # [t, j]: summed over the tokens from t on
    cross = torch.tril(below, -1).sum(-1)
    through = torch.exp(a.sum(-1)) * (G * H).sum((-1, -2))
    d_a = cross + u.flip(-1).cumsum(-1).flip(-1) + (v.cumsum(-1) - v) + through[..., None]
    d_a = d_a.reshape(b, h, -1)[:, :, :s].permute(0, 2, 1)
    d_a = torch.where(f["live"][:, :, None], d_a, 0.0).to(dt).contiguous()
    out = {"y": _unrows(f["y"], case, h, dt), "d_xhat": _unrows(d_x, case, h, dt),
           "d_bhat": _unrows(d_k, case, g, dt), "d_qhat": _unrows(d_q, case, g, dt), "d_da": d_a,
           "d_h0": d_h0 if st["h0"] is not None else None}
    if st["h0"] is not None:
        out["h_last"] = f["last"]
    return out


def _plain_step(st):
    case, state = st["case"], st["state"]
    h, g = case["h"], case["g"]
    used = st["slots"] >= 0
    at = st["slots"].clamp(min=0).long()
    x = st["xhat"][:, 0].float()                                                   # [b,c,h,p]
    k, q = (st[n][:, 0].float().repeat_interleave(h // g, dim=2) for n in ("bhat", "qhat"))
    dec = torch.exp(st["da"][:, 0].float().clamp(min=RESET))[:, :, None, None]     # [b,h,1,1]
    xt = x.permute(0, 2, 3, 1).contiguous()                                        # [b,h,p,c]
    new = state[at] * dec + torch.matmul(xt, k.permute(0, 2, 1, 3).contiguous())
    y = torch.matmul(q.permute(0, 2, 1, 3).contiguous(), new.transpose(-1, -2).contiguous())
    y = torch.where(used[:, None, None, None], y.permute(0, 2, 1, 3), 0.0)
    # by difference, so that the unused rows, which all point at slot 0, leave it as it is
    state.index_add_(0, at, torch.where(used[:, None, None, None], new - state[at], 0.0))
    return {"y": y[:, None].to(st["xhat"].dtype).contiguous(), "state": state}


def _turn(u, rot, kind):
    """The transposed de-rotation of the rows u [b,s,c,h,r]: what brings queries and keys into the cache's frame."""
    if kind == "none":
        return u
    h, r, width = u.shape[3], u.shape[4], rot.shape[3]
    if rot.shape[2] != h:
        rot = rot.repeat_interleave(h // rot.shape[2], dim=2)
    rot = rot.float()[:, :, None]                                                  # one for all channels
    if kind == "quat":
        w, a, b, d = rot.unbind(-1)
        v = u[..., :4 * width].reshape(*u.shape[:4], width, 4)
        v0, v1, v2, v3 = v.unbind(-1)
        a, b, d = -a, -b, -d                                                       # by the conjugate, from the left
        z = torch.stack([w * v0 - a * v1 - b * v2 - d * v3, w * v1 + a * v0 + b * v3 - d * v2,
                         w * v2 - a * v3 + b * v0 + d * v1, w * v3 + a * v2 - b * v1 + d * v0], -1)
        return torch.cat([z.reshape(*u.shape[:4], 4 * width), u[..., 4 * width:]], -1)
    cos, sin = torch.cos(rot), torch.sin(rot)
    if kind == "pairwise":
        v0, v1 = u[..., 0:2 * width:2], u[..., 1:2 * width:2]
        z = torch.stack([v0 * cos - v1 * sin, v0 * sin + v1 * cos], -1).reshape(*u.shape[:4], 2 * width)
        return torch.cat([z, u[..., 2 * width:]], -1)
    n = r // 2
    v0, v1 = u[..., :width], u[..., n:n + width]
    return torch.cat([v0 * cos - v1 * sin, u[..., width:n], v0 * sin + v1 * cos, u[..., n + width:]], -1)


def _plain_norm(st, name):
    case = st["case"]
    x = st[name].float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * rstd
    u = (n * st["w" + name]).repeat_interleave(case["h"] // case["g"], dim=3)
    if st["b" + name] is not None:
        u = u + st["b" + name]
    return n, rstd, u


def _plain_qk(st):
    dt, kind = st["q"].dtype, st["case"]["rot"]
    return {name + "hat": _turn(_plain_norm(st, name)[2], st["rot"], kind).to(dt) for name in ("q", "k")}


def _unturn(z, rot, kind):
    """The de-rotation itself: the transpose of _turn, for cotangents."""
    if kind == "quat":
        return _turn(z, torch.cat([rot[..., :1], -rot[..., 1:]], -1), kind)
    return _turn(z, -rot if rot is not None else None, kind)


def _rot_cotangent(u, z, d, rot, kind):
    """Cotangent of the rotation from one tensor's rows u, its turned rows z and their cotangents d."""
    h, r, width = u.shape[3], u.shape[4], rot.shape[3]
    if kind == "quat":
        cut = lambda t: t[..., :4 * width].reshape(*t.shape[:4], width, 4).unbind(-1)
        u0, u1, u2, u3 = cut(u)
        d0, d1, d2, d3 = cut(d)
        # u times the conjugate of d
        out = torch.stack([u0 * d0 + u1 * d1 + u2 * d2 + u3 * d3, -u0 * d1 + u1 * d0 - u2 * d3 + u3 * d2,
                           -u0 * d2 + u1 * d3 + u2 * d0 - u3 * d1, -u0 * d3 - u1 * d2 + u2 * d1 + u3 * d0], -1)
    elif kind == "pairwise":
        out = z[..., 0:2 * width:2] * d[..., 1:2 * width:2] - z[..., 1:2 * width:2] * d[..., 0:2 * width:2]
    else:
        n = r // 2
        out = z[..., :width] * d[..., n:n + width] - z[..., n:n + width] * d[..., :width]
    out = out.sum(2)                                                               # channels
    hr = rot.shape[2]
    if hr != h:
        out = out.reshape(out.shape[0], out.shape[1], hr, h // hr, *out.shape[3:]).sum(3)
    return out


def _plain_qk_train(st):
    case, dt, kind = st["case"], st["q"].dtype, st["case"]["rot"]
    b, s, c, h, g, r = (case[k] for k in ("b", "s", "c", "h", "g", "r"))
    out, d_rot = {"d_rot": None}, 0.0
    for name in ("q", "k"):
        n, rstd, u = _plain_norm(st, name)
        z = _turn(u, st["rot"], kind)
        d = st["d_%shat" % name].float()
        du = _unturn(d, st["rot"], kind)
        if kind != "none":
            d_rot = d_rot + _rot_cotangent(u, z, d, st["rot"], kind)
        out["d_b" + name] = du.sum((0, 1, 2)) if st["b" + name] is not None else None
        du = du.reshape(b, s, c, g, h // g, r).sum(4)
        out["d_w" + name] = (du * n).sum((0, 1, 2, 3))
        dn = du * st["w" + name]
        out["d_" + name] = ((dn - n * (dn * n).mean(-1, keepdim=True)) * rstd).to(dt)
        out[name + "hat"] = z.to(dt)
    if kind != "none":
        out["d_rot"] = d_rot.to(dt)
    return out


_PLAIN = {"prefill": _plain_prefill, "train": _plain_train, "step": _plain_step, "qk": _plain_qk,
          "qk_train": _plain_qk_train}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("qk", "qk_train"):
        return _exact_qk(st)
    if case["op"] == "step":
        return _exact_step(st)
    return _exact_attn(st)


def _exact_step(st):
    case = st["case"]
    b, c, h, g = case["b"], case["c"], case["h"], case["g"]
    state = st["state"].double()
    y = torch.zeros(b, 1, c, h, case["p"], dtype=torch.float64, device="cuda")
    heads = torch.arange(h, device="cuda") // (h // g)
    for i, slot in enumerate(st["slots"].tolist()):
        if slot < 0:
            continue
        S = state[slot] * torch.exp(st["da"][i, 0].double())[:, None, None]
        for ci in range(c):
            S = S + st["xhat"][i, 0, ci].double()[:, :, None] * st["bhat"][i, 0, ci].double()[heads][:, None, :]
        for ci in range(c):
            y[i, 0, ci] = (S * st["qhat"][i, 0, ci].double()[heads][:, None, :]).sum(-1)
        state[slot] = S
    return {"y": y, "state": state}


def _exact_attn(st):
    """Token by token: the state forwards, its cotangent backwards."""
    case = st["case"]
    b, s, c, h, g, p, r = (case[k] for k in ("b", "s", "c", "h", "g", "p", "r"))
    if s * (2 if case["op"] == "train" else 1) > 70000:
        return None      # over 20 seconds of single tokens
    train = case["op"] == "train"
    n, per = b * h, h // g
    lens = _lens(st)
    live = (torch.arange(s, device="cuda")[None] < lens[:, None])

    def chains(x, heads):                       # [s, b*h, c, w], zero where padding
        x = torch.where(live[:, :, None, None, None], x, 0).double()
        if heads != h:
            x = x.repeat_interleave(per, dim=3)
        return x.permute(1, 0, 3, 2, 4).reshape(s, n, c, -1).contiguous()

    x, k, q = chains(st["xhat"], h), chains(st["bhat"], g), chains(st["qhat"], g)
    dec = torch.exp(torch.where(live[:, :, None], st["da"].double(), 0.0)).permute(1, 0, 2).reshape(s, n, 1, 1)
    H = st["h0"].double().reshape(n, p, r).clone() if st["h0"] is not None else torch.zeros(
        n, p, r, dtype=torch.float64, device="cuda")
    y = torch.empty(s, n, c, p, dtype=torch.float64, device="cuda")
    xt = x.transpose(2, 3).contiguous()
    if train:
        dy = chains(st["d_y"], h)
        dq = torch.empty(s, n, c, r, dtype=torch.float64, device="cuda")
    for t in range(s):
        H.mul_(dec[t]).baddbmm_(xt[t], k[t])
        torch.bmm(q[t], H.transpose(1, 2), out=y[t])
        if train:
            torch.bmm(dy[t], H, out=dq[t])

    def back(z, heads):
        z = z.reshape(s, b, h, c, -1)
        if heads != h:
            z = z.reshape(s, b, heads, per, c, z.shape[-1]).sum(3)
        return z.permute(1, 0, 3, 2, 4)

    out = {"y": back(y, h)}
    if not train:
        out["h_last"] = H.reshape(b, h, p, r)
        return out
    last = H
    G = st["d_h_last"].double().reshape(n, p, r).clone() if st["d_h_last"] is not None else torch.zeros_like(H)
    end = (G * last).sum((1, 2))
    dx, dk = torch.empty_like(y), torch.empty_like(dq)
    dyt = dy.transpose(2, 3).contiguous()
    for t in range(s - 1, -1, -1):
        G.baddbmm_(dyt[t], q[t])
        torch.bmm(k[t], G.transpose(1, 2), out=dx[t])
        torch.bmm(x[t], G, out=dk[t])
        G.mul_(dec[t])
    # every factor exp(da[t]) stands in what the tokens from t on read and in nothing that they write
    per_token = (q * dq).sum((2, 3)) - (k * dk).sum((2, 3))
    d_a = per_token.flip(0).cumsum(0).flip(0) + end
    d_a = torch.where(live[:, :, None], d_a.reshape(s, b, h).permute(1, 0, 2), 0.0)
    if st["h0"] is None:
        d_a[:, 0] = 0.0      # nothing for the first decay to scale; the sums leave the rounding of 64 bits
    out.update(d_xhat=back(dx, h), d_bhat=back(dk, g), d_qhat=back(dq, g), d_da=d_a,
               d_h0=G.reshape(b, h, p, r) if st["h0"] is not None else None)
    if st["h0"] is not None:
        out["h_last"] = last.reshape(b, h, p, r)
    return out


def _exact_qk(st):
    case, kind = st["case"], st["case"]["rot"]
    h, g, r = case["h"], case["g"], case["r"]
    train = case["op"] == "qk_train"
    names = ["q", "k", "wq", "wk", "bq", "bk", "rot"]
    t = {n: None if st[n] is None else st[n].double().contiguous().requires_grad_(train) for n in names}
    M = None
    if kind != "none":                          # the de-rotation as a matrix on each pair or block
        rot = t["rot"].repeat_interleave(h // t["rot"].shape[2], dim=2)
        if kind == "quat":
            w, x, y, z = rot.unbind(-1)
            M = torch.stack([torch.stack([w, -x, -y, -z], -1), torch.stack([x, w, -z, y], -1),
                             torch.stack([y, z, w, -x], -1), torch.stack([z, -y, x, w], -1)], -2)
        else:
            M = torch.stack([torch.stack([rot.cos(), rot.sin()], -1), torch.stack([-rot.sin(), rot.cos()], -1)], -2)
    res = {}
    for n in ("q", "k"):
        x = t[n]
        u = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / r + EPS) * t["w" + n]
        u = u[:, :, :, :, None].expand(-1, -1, -1, -1, h // g, -1).reshape(*u.shape[:3], h, r)
        if t["b" + n] is not None:
            u = u + t["b" + n]
        if M is not None:
            m, width = M.shape[-1], M.shape[3]
            idx = torch.arange(m * width, device="cuda").reshape(width, m)
            if kind == "half":
                i = torch.arange(width, device="cuda")
                idx = torch.stack([i, r // 2 + i], -1)
            v = u[..., idx]                                             # [b,s,c,h,width,m]
            v = (M[:, :, None] * v[..., :, None]).sum(-2)               # by the transpose: columns against rows
            u = u.index_copy(4, idx.reshape(-1), v.reshape(*u.shape[:4], m * width))
        res[n + "hat"] = u
    if not train:
        return res
    have = [n for n in names if t[n] is not None]
    grads = torch.autograd.grad([res["qhat"], res["khat"]], [t[n] for n in have],
                                [st["d_qhat"].double(), st["d_khat"].double()])
    out = {"d_" + n: None for n in names}
    out.update({"d_" + n: v for n, v in zip(have, grads)})
    out.update({n: v.detach() for n, v in res.items()})
    return out


# ------------------------------------------------------------------------------------------------ what it takes
def work(case):
    """Bytes of every input once and every output once; operations of the recurrence: a write and a read of the
    state for each row of the sequence (and their gradients, twice each), the norm and turn of each value."""
    e = 4 if case["dtype"] == "f32" else 2
    b, s, c, h, g, r = (case[k] for k in ("b", "s", "c", "h", "g", "r"))
    if case["op"] in ("qk", "qk_train"):
        rot = b * s * case["rot_h"] * case["width"] * (4 if case["rot"] == "quat" else 1)
        raw, hat = 2 * b * s * c * g * r, 2 * b * s * c * h * r
        param = 4 * 2 * (r + (h * r if case["bias"] else 0))
        if case["op"] == "qk":
            return {"bytes": e * (raw + hat + rot) + param, "flops": 8 * hat}
        return {"bytes": e * (2 * raw + 2 * hat + 2 * rot) + 2 * param, "flops": 30 * hat}
    p = case["p"]
    if case["op"] == "step":
        return {"bytes": b * (8 * h * p * r + e * (2 * c * h * p + 2 * c * g * r + h) + 4),
                "flops": b * h * p * r * (4 * c + 1)}
    rows = b * min(case["valid"], s) * c // (2 if case["ragged"] else 1)     # ragged lengths: half on average
    st = 4 * b * h * p * r * (2 if case["state"] else 1)
    keys, vals, dec = rows * g * r, rows * h * p, rows // c * h
    if case["op"] == "prefill":
        return {"bytes": e * (2 * keys + vals + dec + b * s * c * h * p) + st, "flops": 4 * rows * h * p * r}
    return {"bytes": e * (2 * keys + 2 * vals + dec + 2 * b * s * c * (g * r + h * p) + b * s * h)
            + (2 * st if case["state"] else 0),
            "flops": 12 * rows * h * p * r}
