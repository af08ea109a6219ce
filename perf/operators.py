"""Cases of the layer operators around the recurrences: the short causal convolution, the selective
state space scan (both for prompts, for training and for single tokens) and the block norms.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at
the end), or, where `own` is true, by the framework's calls.  `exact` states the same definitions in
64 bits, by other means: convolutions as sums of shifted copies, recurrences by doubling.

Activations are [batch, tokens, channels]; parameters (taps, rates, norm weights) are 32-bit.  Sizes
are the training layer's (2 sequences of 8192 tokens, 4096 channels, 32 heads of 128) and the decode
workload's (128 sequences) of this repository, with 16 states a channel and 4 taps, and odd ones.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
CH = 4096


def listed():
    return [
        # one generation step of a full batch through the convolution: latency
        dict(name="conv_step", op="conv_step", dtype="bf16", B=128, T=1, D=CH, K=4),
        # one prompt, its channels the first half of a joint projection's rows
        dict(name="conv_prompt", op="conv", dtype="bf16", B=1, T=2047, D=CH, K=4, ragged=False),
        # the training layer's backward
        dict(name="conv_bwd", op="conv_bwd", dtype="bf16", B=2, T=8192, D=CH, K=4, ragged=False),
        # a padded batch of odd sizes in 32 bits
        dict(name="conv_bwd_odd", op="conv_bwd", dtype="f32", B=3, T=777, D=1001, K=3, ragged=True),
        # one generation step of a full batch through the recurrence
        dict(name="scan_step", op="scan_step", dtype="bf16", B=128, T=1, D=CH, N=16, G=1, z=True),
        # one prompt that ends in a state for generation
        dict(name="scan_prompt", op="scan", dtype="bf16", B=1, T=2048, D=CH, N=16, G=1, z=True,
             ragged=False, h0=False),
        # a padded batch of prompts that continue from states; many states, grouped B and C
        dict(name="scan_ragged", op="scan", dtype="bf16", B=4, T=1000, D=2048, N=64, G=4, z=False,
             ragged=True, h0=True),
        # the training layer, forward and backward: the largest
        dict(name="scan_train", op="scan_train", dtype="bf16", B=2, T=8192, D=CH, N=16, G=1, z=True,
             ragged=False, h0=False),
        # odd sizes in 32 bits, gradients of the states too
        dict(name="scan_train_odd", op="scan_train", dtype="f32", B=3, T=511, D=1000, N=8, G=2,
             z=True, ragged=True, h0=True),
        # between two blocks of a generation step: post norm, gate, scale, residual, next norm
        dict(name="norm_step", op="norm", dtype="bf16", B=128, T=1, D=CH, G=1, heads=False,
             full=True),
        # the attention's output by heads: normed a head, gated, laid out as rows
        dict(name="norm_heads", op="norm", dtype="bf16", B=2, T=8192, D=CH, G=32, heads=True,
             full=False),
        # between two blocks, the training layer's backward
        dict(name="norm_bwd", op="norm_bwd", dtype="bf16", B=2, T=8192, D=CH, G=1, heads=False,
             full=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "conv_bwd", "scan_step", "scan", "scan_train", "norm",
                     "norm_bwd"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op.endswith("step"):
        c.update(B=_log(rng, 1, 256), T=1, D=8 * _log(rng, 8, 512))
    else:
        T = _log(rng, 1, 8192)
        c.update(B=rng.randint(1, 4), T=T, D=_log(rng, 64, CH))
        if rng.random() < 0.7:
            c["D"] = -(-c["D"] // 16) * 16
        while c["B"] * c["T"] * c["D"] > 8192 * CH:
            c["B"], c["T"] = max(1, c["B"] // 2), max(1, c["T"] // 2 + c["T"] % 2)
    if op.startswith("conv"):
        c.update(K=rng.randint(2, 4), ragged=rng.random() < 0.4 and c["T"] > 1)
    elif op.startswith("scan"):
        G = rng.choice([1, 1, 2, 4])
        c["D"] = -(-c["D"] // G) * G
        c.update(N=rng.choice([8, 16, 16, 32]) if op == "scan_train" else rng.choice([8, 16, 16, 64]),
                 G=G, z=rng.random() < 0.7, ragged=rng.random() < 0.4 and c["T"] > 1,
                 h0=rng.random() < 0.5)
        while c["B"] * c["T"] * c["D"] * c["N"] > 8192 * CH * 16:
            c["T"] = c["T"] // 2 + c["T"] % 2
    else:
        heads = rng.random() < 0.4
        if heads:
            c["D"] = max(1, c["D"] // 64) * 64
        c.update(G=c["D"] // 64 if heads else 1, heads=heads, full=rng.random() < 0.6)
    return c


# ---- inputs --------------------------------------------------------------------------------
class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def n(self, *s):
        return torch.randn(*s, generator=self.g, device="cuda")

    def u(self, *s):
        return torch.rand(*s, generator=self.g, device="cuda")


def prepare(case, seed):
    r, B, T, D, dt = _Draw(seed), case["B"], case["T"], case["D"], DT[case["dtype"]]
    st = dict(case=case)
    if case.get("ragged"):
        st["lens"] = (r.u(B) * (T + 1)).long().clamp(max=T)  # a length may be 0 or 1
        st["lens"][0] = T
    op = case["op"]
    if op.startswith("conv"):
        K = case["K"]
        st.update(w=r.n(D, K) / math.sqrt(K), bias=0.1 * r.n(D))
        if op == "conv_step":
            st.update(hist=r.n(B, K - 1, D).to(dt), x=r.n(B, D).to(dt))
        else:  # the channels x of the rows [x | z] that one projection writes
            st.update(x=r.n(B, T, 2 * D).to(dt)[..., :D], x0=r.n(B, K - 1, D).to(dt))
        if op == "conv_bwd":
            st.update(dy=r.n(B, T, D).to(dt))
    elif op.startswith("scan"):
        N, G = case["N"], case["G"]
        # rates -1 .. -N and steps of 0.001 to 0.1, as such layers start out
        delta = torch.exp(r.u(D) * math.log(100.0) + math.log(1e-3))
        st.update(A=-torch.arange(1, N + 1, device="cuda").float() * torch.exp(0.1 * r.n(D, N)),
                  dt_bias=delta + torch.log(-torch.expm1(-delta)), Dskip=1 + 0.1 * r.n(D))
        rows = (B,) if op == "scan_step" else (B, T)
        u = r.n(*rows, D)
        st.update(u=(u * torch.sigmoid(u)).to(dt), dt=(0.5 * r.n(*rows, D)).to(dt))
        bc = r.n(*rows, 2, G, N).to(dt)  # B and C lie side by side in one projection's rows
        st.update(Bm=bc.select(-3, 0), Cm=bc.select(-3, 1))
        if case["z"]:
            st["z"] = r.n(*rows, D).to(dt)
        if case.get("h0") or op == "scan_step":
            st["h0"] = 0.1 * r.n(B, D, N)
        if op == "scan_train":
            st["dy"] = r.n(B, T, D).to(dt)
            if case["h0"]:
                st["dhT"] = 0.1 * r.n(B, D, N)
    else:
        G = case["G"]
        o = r.n(B, G, T, D // G) if case["heads"] else r.n(B, T, D)
        st.update(o=o.to(dt), w=1 + 0.1 * r.n(D), z=r.n(B, T, D).to(dt))
        if case["full"]:
            st.update(s=0.5 + 0.1 * r.n(D), r=r.n(B, T, D).to(dt), w2=1 + 0.1 * r.n(D))
        if op == "norm_bwd":
            with torch.no_grad():  # what the forward left: the residual stream
                st["out"] = _plain_norm(st)[0]
            st["dout"] = r.n(B, T, D).to(dt)
            if case["full"]:
                st["dn"] = r.n(B, T, D).to(dt)
    return st


def work(case):
    B, T, D, es, op = case["B"], case["T"], case["D"], ES[case["dtype"]], case["op"]
    e = B * T * D
    if op.startswith("conv"):
        K = case["K"]
        par, hist = 4 * D * (K + 1), B * D * (K - 1) * es
        if op == "conv_bwd":
            return {"bytes": 3 * e * es + 2 * par + 2 * hist, "flops": e * (6 * K + 10)}
        return {"bytes": 2 * e * es + par + 2 * hist, "flops": e * (2 * K + 4)}
    if op.startswith("scan"):
        N, G, z = case["N"], case["G"], int(case["z"])
        par, hs, bc = 4 * D * (N + 2), 4 * B * D * N, 2 * B * T * G * N * es
        if op == "scan_train":
            return {"bytes": (6 + 2 * z) * e * es + 2 * bc + 2 * par + 4 * int(case["h0"]) * hs,
                    "flops": e * (N * 25 + 30)}
        nh = 1 + int(bool(case.get("h0")) or op == "scan_step")
        return {"bytes": (3 + z) * e * es + bc + par + nh * hs, "flops": e * (N * 7 + 12)}
    f = int(case["full"])
    if op == "norm_bwd":
        return {"bytes": ((4 + 4 * f + 1 - f) * e) * es + 8 * D * (1 + 2 * f), "flops": e * (20 + 15 * f)}
    return {"bytes": (3 + 2 * f) * e * es + 4 * D * (1 + 2 * f), "flops": e * (9 + 6 * f)}


# ---- one pass ------------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    return (_OWN if own else _PLAIN)[op](st)


def _mask(lens, T):
    return (torch.arange(T, device="cuda") < lens[:, None])[..., None]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    s = 1 / (1 + torch.exp(-x))
    return s * (1 + x * (1 - s))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _padded(st):
    """The tokens with the history in front, in 32 bits; nothing behind a sequence's end."""
    x = st["x"].float()
    if "lens" in st:
        x = torch.where(_mask(st["lens"], x.shape[1]), x, torch.zeros_like(x))
    return torch.cat([st["x0"].float(), x], 1)


def _plain_conv_pre(st):
    K, T = st["case"]["K"], st["case"]["T"]
    x = _padded(st)
    p = st["bias"] + st["w"][:, 0] * x[:, :T]
    for j in range(1, K):
        p = p + st["w"][:, j] * x[:, j:j + T]
    return x, p


def _plain_conv(st):
    K, T, dt = st["case"]["K"], st["case"]["T"], st["x"].dtype
    x, p = _plain_conv_pre(st)
    y = _silu(p)
    if "lens" not in st:
        return y.to(dt), x[:, T:].to(dt)
    y = torch.where(_mask(st["lens"], T), y, torch.zeros_like(y))
    at = st["lens"][:, None] + torch.arange(K - 1, device="cuda")
    return y.to(dt), torch.gather(x, 1, at[..., None].expand(-1, -1, x.shape[2])).to(dt)


def _plain_conv_bwd(st):
    K, T, dt = st["case"]["K"], st["case"]["T"], st["x"].dtype
    x, p = _plain_conv_pre(st)
    dp = st["dy"].float() * _dsilu(p)
    if "lens" in st:
        dp = torch.where(_mask(st["lens"], T), dp, torch.zeros_like(dp))
    dx = torch.zeros_like(x)
    dw = torch.empty_like(st["w"])
    for j in range(K):
        dx[:, j:j + T] += st["w"][:, j] * dp
        dw[:, j] = (dp * x[:, j:j + T]).sum(1).sum(0)
    d0 = dx[:, :K - 1]
    dx = dx[:, K - 1:]
    return dx.to(dt), dw, dp.sum(1).sum(0), d0.to(dt)


def _plain_conv_step(st):
    x = torch.cat([st["hist"], st["x"][:, None]], 1)
    p = st["bias"] + (x.float() * st["w"].t()).sum(1)
    st["hist"].copy_(x[:, 1:])
    return _silu(p).to(st["x"].dtype), st["hist"]


def _delta(st):
    d = st["dt"].float() + st["dt_bias"]
    return d, _softplus(d)


def _bc(m, D):
    """[.., G, N] -> [.., D, N], a group's row for each of its channels."""
    return m.float().repeat_interleave(D // m.shape[-2], dim=-2)


def _plain_step(st):
    D = st["case"]["D"]
    u, h = st["u"].float(), st["h0"]
    _, delta = _delta(st)
    h.copy_(torch.exp(delta[..., None] * st["A"]) * h + (delta * u)[..., None] * _bc(st["Bm"], D))
    y = (h * _bc(st["Cm"], D)).sum(-1) + st["Dskip"] * u
    if "z" in st:
        y = y * _silu(st["z"].float())
    return y.to(st["u"].dtype), h


CHUNK = 1024  # tokens that are expanded to [tokens, batch, channels, states] at a time


def _expand(st, delta, u, t0, t1, keep):
    """Decays and inputs of tokens t0..t1, [tokens, batch, channels, states]; a token behind its
    sequence's end keeps the state."""
    D = st["case"]["D"]
    dl = delta[:, t0:t1].transpose(0, 1)
    if keep is not None:
        dl = dl * keep[:, t0:t1].transpose(0, 1)
    a = torch.exp(dl[..., None] * st["A"])
    b = (dl * u[:, t0:t1].transpose(0, 1))[..., None] * _bc(st["Bm"][:, t0:t1], D).transpose(0, 1)
    return a, b


def _plain_scan(st, states=None):
    c = st["case"]
    B, T, D, N = (c[k] for k in "BTDN")
    u, keep = st["u"].float(), None
    _, delta = _delta(st)
    if "lens" in st:
        keep = _mask(st["lens"], T)
        u = torch.where(keep, u, torch.zeros_like(u))
    h = st["h0"].clone() if "h0" in st else torch.zeros(B, D, N, device="cuda")
    y = torch.empty(B, T, D, device="cuda")
    for t0 in range(0, T, CHUNK):
        t1 = min(T, t0 + CHUNK)
        a, b = _expand(st, delta, u, t0, t1, keep)
        if states is not None:
            states.append(h)
        for t in range(t1 - t0):
            h = torch.addcmul(b[t], a[t], h, out=b[t])
        h = h.clone()
        y[:, t0:t1] = (b * _bc(st["Cm"][:, t0:t1], D).transpose(0, 1)).sum(-1).transpose(0, 1)
    raw = y + st["Dskip"] * u
    y = raw * _silu(st["z"].float()) if "z" in st else raw
    if keep is not None:
        y = torch.where(keep, y, torch.zeros_like(y))
    return y.to(st["u"].dtype), h, raw


def _plain_scan_train(st):
    c = st["case"]
    B, T, D, N, G = (c[k] for k in "BTDNG")
    dt, states = st["u"].dtype, []
    y, hT, raw = _plain_scan(st, states)
    u, dy, keep = st["u"].float(), st["dy"].float(), None
    pre, delta = _delta(st)
    if "lens" in st:
        keep = _mask(st["lens"], T)
        u, dy = (torch.where(keep, x, torch.zeros_like(x)) for x in (u, dy))
    out = {"y": y, "hT": hT}
    e = dy
    if "z" in st:
        z = st["z"].float()
        e = dy * _silu(z)
        out["dz"] = (dy * raw * _dsilu(z)).to(dt)
    dskip = (e * u).sum(1).sum(0)
    du, ddelta = st["Dskip"] * e, torch.zeros_like(e)
    dA = torch.zeros(D, N, device="cuda")
    dB, dC = (torch.zeros(B, T, G, N, device="cuda") for _ in range(2))
    g = st["dhT"].clone() if "dhT" in st else torch.zeros(B, D, N, device="cuda")
    for i in reversed(range(len(states))):
        t0, t1 = i * CHUNK, min(T, i * CHUNK + CHUNK)
        n = t1 - t0
        a, h = _expand(st, delta, u, t0, t1, keep)
        s = states[i]
        for t in range(n):
            s = torch.addcmul(h[t], a[t], s, out=h[t])
        ee, dl, uu = (x[:, t0:t1].transpose(0, 1)[..., None] for x in (e, delta, u))
        grp = lambda x: x.reshape(n, B, G, D // G, N).sum(3).transpose(0, 1)
        dC[:, t0:t1] = grp(ee * h)
        p = torch.cat([states[i][None], h[:-1]]) * a  # decay x state before the token
        del h
        Bx = _bc(st["Bm"][:, t0:t1], D).transpose(0, 1)
        gs = ee * _bc(st["Cm"][:, t0:t1], D).transpose(0, 1)
        for t in reversed(range(n)):  # gs[t] becomes the gradient of the state after token t
            g = torch.addcmul(gs[t], a[t + 1], g, out=gs[t]) if t + 1 < n else gs[t].add_(g)
        dB[:, t0:t1] = grp(gs * (dl * uu))
        gB = (gs * Bx).sum(-1)
        du[:, t0:t1] += (gB * dl[..., 0]).transpose(0, 1)
        p *= gs
        g = gs[0] * a[0]
        pd = p * dl if keep is None else p * (dl * keep[:, t0:t1].transpose(0, 1)[..., None])
        dA += pd.sum(0).sum(0)
        ddelta[:, t0:t1] = (gB * uu[..., 0] + (p * st["A"]).sum(-1)).transpose(0, 1)
    if keep is not None:
        ddelta = torch.where(keep, ddelta, torch.zeros_like(ddelta))
        du = torch.where(keep, du, torch.zeros_like(du))
    ddt = ddelta / (1 + torch.exp(-pre))
    out.update(du=du.to(dt), ddt=ddt.to(dt), dA=dA, dB=dB.to(dt), dC=dC.to(dt), dDskip=dskip,
               ddt_bias=ddt.sum(1).sum(0))
    if c["h0"]:
        out["dh0"] = g
    return out


EPS = 1e-5


def _rows(o):
    """[batch, heads, tokens, features] -> rows."""
    return o.transpose(1, 2).reshape(o.shape[0], o.shape[2], -1) if o.dim() == 4 else o


def _plain_norm(st):
    c, dt = st["case"], st["o"].dtype
    o = _rows(st["o"].float())
    grp = o.view(*o.shape[:2], c["G"], -1)
    m = (grp * torch.rsqrt((grp * grp).mean(-1, keepdim=True) + EPS)).view_as(o) * st["w"]
    m = m * _silu(st["z"].float())
    if not c["full"]:
        return (m.to(dt),)
    out = (st["r"].float() + st["s"] * m).to(dt)
    x = out.float()
    return out, (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * st["w2"]).to(dt)


def _plain_norm_bwd(st):
    c, dt = st["case"], st["o"].dtype
    B, T, D, G = (c[k] for k in "BTDG")
    e, res = st["dout"].float(), {}
    if c["full"]:
        x, dn = st["out"].float(), st["dn"].float()
        rs = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * rs
        res["dw2"] = (dn * xh).sum(1).sum(0)
        q = dn * st["w2"]
        e = e + rs * (q - xh * (q * xh).mean(-1, keepdim=True))
        res["dr"] = e.to(dt)
    o = _rows(st["o"].float()).view(B, T, G, -1)
    rs = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)
    mh = (o * rs).view(B, T, D)
    z = st["z"].float()
    core, sz = mh * st["w"], _silu(z)
    if c["full"]:
        res["ds"] = (e * core * sz).sum(1).sum(0)
        e = e * st["s"]
    res["dz"] = (e * core * _dsilu(z)).to(dt)
    e = e * sz
    res["dw"] = (e * mh).sum(1).sum(0)
    q, mh = (e * st["w"]).view(B, T, G, -1), mh.view(B, T, G, -1)
    do = rs * (q - mh * (q * mh).mean(-1, keepdim=True))
    res["do"] = (do.transpose(1, 2).contiguous() if c["heads"] else do.reshape(B, T, D)).to(dt)
    return res


# ---- the framework's calls -----------------------------------------------------------------
def _lib():
    import gated_linear_sliding_chunked_b200 as L
    return L


def _own_conv(st):
    return _lib().conv_fwd(st["x"], st["w"], st["bias"], st["x0"], lens=st.get("lens"), want_xT=True)


def _own_conv_bwd(st):
    d = _lib().conv_bwd(st["x"], st["w"], st["dy"], st["bias"], st["x0"], lens=st.get("lens"),
                        want_dx0=True)
    return d["dx"], d["dw"], d["dbias"], d["dx0"]


def _own_conv_step(st):
    return _lib().conv_step(st["hist"], st["x"], st["w"], st["bias"]), st["hist"]


def _scan_kw(st, *more):
    return {k: st.get(k) for k in ("Dskip", "z", "dt_bias") + more}


def _own_step(st):
    y = _lib().scan_step(st["h0"], *(st[k] for k in ("u", "dt", "A", "Bm", "Cm")), **_scan_kw(st))
    return y, st["h0"]


def _own_scan(st):
    return _lib().scan_fwd(*(st[k] for k in ("u", "dt", "A", "Bm", "Cm")),
                           **_scan_kw(st, "h0", "lens"), want_hT=True)


def _own_scan_train(st):
    L, a = _lib(), [st[k] for k in ("u", "dt", "A", "Bm", "Cm")]
    y, hT, states = L.scan_fwd(*a, **_scan_kw(st, "h0", "lens"), want_hT=True, want_states=True)
    d = L.scan_bwd(*a, st["dy"], **_scan_kw(st, "h0", "lens", "dhT"), states=states,
                   want_dh0=st["case"]["h0"])
    out = {"y": y, "hT": hT}
    if "z" in st:
        out["dz"] = d["dz"]
    out.update({k: d[k] for k in ("du", "ddt", "dA", "dB", "dC", "dDskip", "ddt_bias")})
    if st["case"]["h0"]:
        out["dh0"] = d["dh0"]
    return out


def _norm_kw(st, *more):
    kw = {k: st.get(k) for k in ("w", "z", "s", "w2") + more}
    return dict(kw, groups=st["case"]["G"], eps=EPS)


def _own_norm(st):
    out, n = _lib().block_norm_fwd(st["o"], **_norm_kw(st, "r"))
    return (out, n) if st["case"]["full"] else (out,)


def _own_norm_bwd(st):
    d = _lib().block_norm_bwd(st["o"], **_norm_kw(st, "dout", "dn"),
                              out=st["out"] if st["case"]["full"] else None,
                              want_dr=st["case"]["full"])
    names = ("dw2", "dr", "ds", "dz", "dw", "do") if st["case"]["full"] else ("dz", "dw", "do")
    return {k: d[k] for k in names}


_PLAIN = dict(conv_step=_plain_conv_step, conv=_plain_conv, conv_bwd=_plain_conv_bwd,
              scan_step=_plain_step, scan=lambda st: _plain_scan(st)[:2],
              scan_train=_plain_scan_train, norm=_plain_norm, norm_bwd=_plain_norm_bwd)
_OWN = dict(conv_step=_own_conv_step, conv=_own_conv, conv_bwd=_own_conv_bwd, scan_step=_own_step,
            scan=_own_scan, scan_train=_own_scan_train, norm=_own_norm, norm_bwd=_own_norm_bwd)


# ---- the definitions in 64 bits ------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    st = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
          for k, v in st.items()}
    op = case["op"]
    if op.startswith("conv"):
        return _exact_conv(case, st)
    if op.startswith("scan"):
        return _exact_scan(case, st)
    return _exact_norm(case, st)


def _sig(x):
    return torch.sigmoid(x)


def _ends(case, st):
    return [int(x) for x in st["lens"]] if "lens" in st else [case["T"]] * case["B"]


def _exact_conv(case, st):
    K, T, B, D = (case[k] for k in "KTBD")
    w = st["w"]
    if case["op"] == "conv_step":
        p = st["bias"] + w[:, K - 1] * st["x"]
        for j in range(K - 1):
            p = p + w[:, j] * st["hist"][:, j]
        return p * _sig(p), torch.cat([st["hist"], st["x"][:, None]], 1)[:, 1:]
    rows, last = [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(st["bias"])
    for b, n in enumerate(_ends(case, st)):
        x = torch.cat([st["x0"][b], st["x"][b, :n]])
        win = x.unfold(0, K, 1) if n else x.new_zeros(0, D, K)
        p = (win * w).sum(-1) + st["bias"]
        if case["op"] == "conv":
            rows.append(torch.cat([p * _sig(p), p.new_zeros(T - n, D)]))
            last.append(x[n:])
            continue
        s = _sig(p)
        dp = st["dy"][b, :n] * (s + p * s * (1 - s))
        dw += (win * dp[..., None]).sum(0)
        db += dp.sum(0)
        dx = sum(torch.cat([x.new_zeros(j, D), dp * w[:, j], x.new_zeros(K - 1 - j, D)])
                 for j in range(K))
        last.append(dx[:K - 1])
        rows.append(torch.cat([dx[K - 1:], x.new_zeros(T - n, D)]))
    if case["op"] == "conv":
        return torch.stack(rows), torch.stack(last)
    return torch.stack(rows), dw, db, torch.stack(last)


def _doubled(a, b):
    """x_t = a_t x_{t-1} + b_t along the first axis, from x_{-1} = 0, by doubling."""
    a, b, s = a.clone(), b.clone(), 1
    while s < len(a):
        b[s:] += a[s:] * b[:-s].clone()
        a[s:] *= a[:-s].clone()
        s *= 2
    return b


def _exact_scan(case, st):
    B, T, D, N, G = (case[k] for k in "BTDNG")
    A, per, op = st["A"], D // G, case["op"]
    pre = st["dt"] + st["dt_bias"]
    delta = torch.logaddexp(pre, torch.zeros_like(pre))
    if op == "scan_step":
        Bx, Cx = (st[k].repeat_interleave(per, 1) for k in ("Bm", "Cm"))
        h = torch.exp(delta[..., None] * A) * st["h0"] + (delta * st["u"])[..., None] * Bx
        y = (h * Cx).sum(-1) + st["Dskip"] * st["u"]
        return (y * st["z"] * _sig(st["z"]) if "z" in st else y), h
    y = torch.zeros(B, T, D, device="cuda", dtype=torch.float64)
    hT = torch.zeros(B, D, N, device="cuda", dtype=torch.float64)
    gr = {k: torch.zeros_like(y) for k in ("du", "ddt", "dz")}
    gr.update(dA=torch.zeros_like(A), dDskip=A.new_zeros(D), ddt_bias=A.new_zeros(D),
              dB=A.new_zeros(B, T, G, N), dC=A.new_zeros(B, T, G, N), dh0=torch.zeros_like(hT))
    for b, n in enumerate(_ends(case, st)):
        for lo in range(0, D, 512):  # blocks of channels: [tokens, channels, states] at a time
            ch = torch.arange(lo, min(D, lo + 512), device="cuda")
            h0 = st["h0"][b, ch] if "h0" in st else A.new_zeros(len(ch), N)
            dhT = st["dhT"][b, ch] if "dhT" in st else A.new_zeros(len(ch), N)
            if n == 0:
                hT[b, ch], gr["dh0"][b, ch] = h0, dhT
                continue
            dl, u = delta[b, :n, ch], st["u"][b, :n, ch]
            Bx, Cx = (st[k][b, :n, ch // per] for k in ("Bm", "Cm"))
            a = torch.exp(dl[..., None] * A[ch])
            x = (dl * u)[..., None] * Bx
            x[0] += a[0] * h0
            h = _doubled(a, x)
            raw = (h * Cx).sum(-1) + st["Dskip"][ch] * u
            z = st["z"][b, :n, ch] if "z" in st else None
            gate = z * _sig(z) if z is not None else torch.ones_like(raw)
            y[b, :n, ch], hT[b, ch] = raw * gate, h[-1]
            if op == "scan":
                continue
            dy = st["dy"][b, :n, ch]
            e = dy * gate
            if z is not None:
                gr["dz"][b, :n, ch] = dy * raw * _sig(z) * (1 + z - z * _sig(z))
            x = e[..., None] * Cx
            x[-1] += dhT
            # from the last token to the first: g_t = x_t + a_{t+1} g_{t+1}
            g = _doubled(torch.cat([A.new_zeros(1, len(ch), N), a.flip(0)[:-1]]), x.flip(0)).flip(0)
            ga = g * a * torch.cat([h0[None], h[:-1]])
            gB = (g * Bx).sum(-1)
            dd = (gB * u + (ga * A[ch]).sum(-1)) * _sig(pre[b, :n, ch])
            gr["du"][b, :n, ch] = gB * dl + st["Dskip"][ch] * e
            gr["ddt"][b, :n, ch] = dd
            gr["dA"][ch] += (ga * dl[..., None]).sum(0)
            gr["dDskip"][ch] += (e * u).sum(0)
            gr["ddt_bias"][ch] += dd.sum(0)
            gr["dh0"][b, ch] = g[0] * a[0]
            gr["dB"][b, :n].index_add_(1, ch // per, g * (dl * u)[..., None])
            gr["dC"][b, :n].index_add_(1, ch // per, h * e[..., None])
    if op == "scan":
        return y, hT
    out = {"y": y, "hT": hT}
    if "z" in st:
        out["dz"] = gr["dz"]
    out.update({k: gr[k] for k in ("du", "ddt", "dA", "dB", "dC", "dDskip", "ddt_bias")})
    if case["h0"]:
        out["dh0"] = gr["dh0"]
    return out


def _exact_norm(case, st):
    B, T, D, G = (case[k] for k in "BTDG")
    o = st["o"].permute(0, 2, 1, 3).reshape(B, T, D) if case["heads"] else st["o"]

    def unit(x, groups):  # each group divided by its root mean square, with that factor
        x = x.reshape(B, T, groups, D // groups)
        f = 1 / torch.sqrt(x.pow(2).sum(-1, keepdim=True) * (groups / D) + EPS)
        return (x * f).reshape(B, T, D), f

    def unit_grad(q, x, f, groups):
        q, x = (v.reshape(B, T, groups, D // groups) for v in (q, x))
        return (f * (q - x * (q * x).sum(-1, keepdim=True) * (groups / D))).reshape(B, T, D)

    m, f = unit(o, G)
    gate = st["z"] * _sig(st["z"])
    if case["op"] == "norm":
        y = m * st["w"] * gate
        if not case["full"]:
            return (y,)
        out = st["r"] + y * st["s"]
        # the second norm reads the stored stream: its own rounding of `out` is part of it
        return out, unit(out.to(DT[case["dtype"]]).double(), 1)[0] * st["w2"]
    e, res = st["dout"], {}
    s = st["s"] if case["full"] else torch.ones_like(st["w"])
    if case["full"]:
        x, fx = unit(st["out"], 1)
        res["dw2"] = torch.einsum("btd,btd->d", st["dn"], x)
        e = e + unit_grad(st["dn"] * st["w2"], x, fx, 1)
        res["dr"] = e
        res["ds"] = torch.einsum("btd,btd->d", e, m * st["w"] * gate)
    sg = _sig(st["z"])
    res["dz"] = e * s * m * st["w"] * (sg + gate * (1 - sg))
    res["dw"] = torch.einsum("btd,btd->d", e * s * gate, m)
    do = unit_grad(e * s * gate * st["w"], m, f, G)
    res["do"] = (do.reshape(B, T, G, D // G).permute(0, 2, 1, 3).contiguous() if case["heads"]
                 else do)
    return res
