"""The layer operators (short convolution, selective scan, block norms) from
their definitions in 64 bits (numpy), with their gradients by formula, and the
bounds that the GPU tests hold the kernels to.

Bounds.  A kernel's result is off by the rounding of the stored value, at most
half a step of its type relative to the value, and by the roundings on the way,
each at most 2^-24 relative to an intermediate (exponentials, logarithms and
quotients: a few of these).  An intermediate is at most its majorant, the same
formula with every term replaced by its absolute value; so a result of at most
k roundings in sequence is within  half * |ref| + k 2^-24 * majorant.  Every
function takes absval=True to evaluate the majorant.
"""
import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U32 = 2.0 ** -24


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def check(name, got, ref, maj, k, dtype):
    """|got - ref| <= half |ref| + k 2^-24 maj, element by element."""
    got = np64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    # the bound on the rounding counts from the value that was rounded
    tol = (HALF[dtype] * np.abs(ref) + k * U32 * maj) * (1 + 2.0 ** -7) + 1e-37
    err = np.abs(got - ref)
    bad = err > tol
    if bad.any():
        i = np.unravel_index(np.argmax(err / tol), err.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} out of bounds, worst at {i}: got "
                             f"{got[i]:.9g}, ref {ref[i]:.9g}, err {err[i]:.3g}, tol {tol[i]:.3g}")


def sig(x):
    return 0.5 * (1 + np.tanh(0.5 * x))


def silu(x, absval=False):
    y = x * sig(x)
    return np.abs(y) if absval else y


def dsilu(x, absval=False):
    s = sig(x)
    # the derivative's two terms, of either sign
    return s + np.abs(x) * s * (1 - s) if absval else s * (1 + x * (1 - s))


def _a(absval):
    return (lambda x: None if x is None else np.abs(x)) if absval else (lambda x: x)


def _lens(lens, B, T):
    return [T] * B if lens is None else [int(min(max(n, 0), T)) for n in lens]


# ---- convolution ------------------------------------------------------------
def _conv_pre(x, w, bias, x0):
    """Tokens with history [K-1+n, D] and p [n, D] of one sequence."""
    K = w.shape[1]
    xx = np.concatenate([x0, x]) if K > 1 else x
    n = len(x)
    p = np.broadcast_to(bias, (n, x.shape[1])).copy()
    for j in range(K):
        p += w[:, j] * xx[j:j + n]
    return xx, p


def conv(x, w, bias=None, x0=None, lens=None, act=True, dy=None, dxT=None, absval=False):
    """dict(y, xT) and, with dy, dx, dw, dbias, dx0.  The majorant of act(p) is
    that of its argument's error carried on: |act'| <= 1.1, plus |y|."""
    a = _a(absval)
    (B, T, D), K = x.shape, w.shape[1]
    bias = np.zeros(D) if bias is None else bias
    x0 = np.zeros((B, K - 1, D)) if x0 is None else x0
    out = {"y": np.zeros((B, T, D)), "xT": np.zeros((B, K - 1, D))}
    if dy is not None:
        out.update(dx=np.zeros((B, T, D)), dw=np.zeros((D, K)), dbias=np.zeros(D),
                   dx0=np.zeros((B, K - 1, D)))
    for b, n in enumerate(_lens(lens, B, T)):
        xx, p = _conv_pre(x[b, :n], w, bias, x0[b])
        mp = _conv_pre(a(x[b, :n]), a(w), a(bias), a(x0[b]))[1] if absval else p
        out["y"][b, :n] = (1.1 * mp + np.abs(silu(p)) if absval else silu(p)) if act else mp
        out["xT"][b] = xx[n:]
        if dy is None:
            continue
        d = a(dy[b, :n])
        if act:  # |silu''| <= 1/2 carries the argument's error on
            d = d * (dsilu(p, True) + 0.5 * mp if absval else dsilu(p))
        dxx = np.zeros((n + K - 1, D))
        for j in range(K):
            dxx[j:j + n] += a(w[:, j]) * d
            out["dw"][:, j] += (d * a(xx[j:j + n])).sum(0)
        out["dbias"] += d.sum(0)
        if dxT is not None:
            dxx[n:] += a(dxT[b])
        out["dx0"][b] = dxx[:K - 1]
        out["dx"][b, :n] = dxx[K - 1:]
    return out


# ---- selective scan ---------------------------------------------------------
def scan(u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, softplus=True, h0=None, lens=None,
         dy=None, dhT=None, absval=False):
    """dict(y, hT) and, with dy, every gradient.  u, dt, z [B,T,D]; Bm, Cm
    [B,T,G,N]."""
    a = _a(absval)
    B, T, D = u.shape
    G, N = Bm.shape[2:]
    grp = np.arange(D) // (D // G)
    zero = np.zeros(D)
    Dskip = a(zero if Dskip is None else Dskip)
    pre = dt + (zero if dt_bias is None else dt_bias)
    delta = np.logaddexp(pre, 0) if softplus else pre
    dsp = sig(pre) if softplus else np.ones_like(pre)
    # a step's own error, relative to the step's majorant |dt| + |bias|
    md = delta
    if absval:
        mpre = np.abs(dt) + np.abs(zero if dt_bias is None else dt_bias)
        md = np.abs(delta) + dsp * mpre
    u, Bm, Cm, dy, dhT, Am = a(u), a(Bm), a(Cm), a(dy), a(dhT), a(A)
    h0 = np.zeros((B, D, N)) if h0 is None else a(h0)
    gate = np.ones_like(pre) if z is None else silu(z, absval)
    out = {"y": np.zeros((B, T, D)), "hT": np.zeros((B, D, N))}
    if dy is not None:
        out.update(du=np.zeros((B, T, D)), ddt=np.zeros((B, T, D)), dA=np.zeros((D, N)),
                   dB=np.zeros((B, T, G, N)), dC=np.zeros((B, T, G, N)), dDskip=np.zeros(D),
                   ddt_bias=np.zeros(D), dh0=np.zeros((B, D, N)))
        if z is not None:
            out["dz"] = np.zeros((B, T, D))
    for b, n in enumerate(_lens(lens, B, T)):
        h = h0[b]
        H, P, AL = [h], [], []
        for t in range(n):
            al = np.exp(delta[b, t, :, None] * A)
            P.append(al * h)
            h = P[-1] + (md[b, t] * u[b, t])[:, None] * Bm[b, t][grp]
            AL.append(al)
            H.append(h)
            raw = (h * Cm[b, t][grp]).sum(1) + Dskip * u[b, t]
            out["y"][b, t] = raw * gate[b, t]
            if dy is not None and z is not None:
                out["dz"][b, t] = dy[b, t] * raw * dsilu(z[b, t], absval)
        out["hT"][b] = h
        if dy is None:
            continue
        g = np.zeros((D, N)) if dhT is None else dhT[b]
        for t in range(n - 1, -1, -1):
            e = dy[b, t] * gate[b, t]
            Bg, Cg = Bm[b, t][grp], Cm[b, t][grp]
            g = g + e[:, None] * Cg
            np.add.at(out["dC"][b, t], grp, e[:, None] * H[t + 1])
            np.add.at(out["dB"][b, t], grp, g * (md[b, t] * u[b, t])[:, None])
            gB = (g * Bg).sum(1)
            gp = g * P[t]
            out["dA"] += gp * md[b, t][:, None]
            dd = (u[b, t] * gB + (gp * Am).sum(1)) * dsp[b, t]
            out["ddt"][b, t] = dd
            out["ddt_bias"] += dd
            out["du"][b, t] = md[b, t] * gB + Dskip * e
            out["dDskip"] += e * u[b, t]
            g = g * AL[t]
        out["dh0"][b] = g
    return out


# ---- block norms ------------------------------------------------------------
def _unit(x, G, eps):
    """rmsnorm over G runs of features: normed rows, 1/rms broadcast."""
    y = x.reshape(*x.shape[:-1], G, -1)
    rs = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    return (y * rs).reshape(x.shape), np.broadcast_to(rs, y.shape).reshape(x.shape)


def _unit_grad(q, xh, rs, G, absval):
    y = (q * xh).reshape(*q.shape[:-1], G, -1)
    m = np.broadcast_to(y.mean(-1, keepdims=True), y.shape).reshape(q.shape)
    return rs * (q + xh * m if absval else q - xh * m)


def norm(o, w=None, z=None, s=None, r=None, w2=None, groups=1, eps=1e-5, out=None, dout=None,
         dn=None, absval=False):
    """dict(out, n) for rows o [B,T,D] and, with dout or dn (and the stored
    `out`), the gradients.  With a stored `out`, n is that of it."""
    a = _a(absval)
    one = np.ones(o.shape[-1])
    mh, rs = (o, np.ones_like(o)) if w is None else _unit(o, groups, eps)
    core = a(mh) * a(one if w is None else w)
    gate = np.ones_like(o) if z is None else silu(z, absval)
    sv = a(one if s is None else s)
    res = {"out": core * gate * sv + (0 if r is None else a(r))}
    stored = res["out"] if out is None else out
    if w2 is not None:
        xh, rs2 = _unit(stored, 1, eps)
        xh = a(xh)
        res["n"] = xh * a(w2)
    if dout is None and dn is None:
        return res
    e = 0 if dout is None else a(dout)
    if dn is not None:
        q = a(dn) * a(w2)
        e = e + _unit_grad(q, xh, rs2, 1, absval)
        res["dw2"] = (a(dn) * xh).sum((0, 1))
    mh = a(mh)
    res["dr"] = e
    res["ds"] = (e * core * gate).sum((0, 1))
    f = e * sv
    if z is not None:
        res["dz"] = f * core * dsilu(z, absval)
    f = f * gate
    res["dw"] = (f * mh).sum((0, 1))
    k = f * a(one if w is None else w)
    res["do"] = k if w is None else _unit_grad(k, mh, rs, groups, absval)
    return res
