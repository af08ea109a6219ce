"""The selective scan in 64 bits (numpy) with a running bound on what 32-bit arithmetic may be off by.

Every quantity carries its own error along: a sum or product adds one rounding, 2^-24 of its value,
to what its operands are off by, and a state's error decays with the state.  So a bound is a few
2^-24 of the values that really meet in it, times the memory of the state, not a worst case over the
whole sequence.  First order only (5 % on top).  The functions' own errors, relative (u = 2^-24):
2^x 4 u (the documented bound of ex2.approx), 1/x 2 u (rcp.approx), and what they pass on."""
import numpy as np

U = 2.0 ** -24
EX = 4.2 * U  # 2^x, with the constant in its exponent


def _sig(x):
    return 0.5 * (1 + np.tanh(0.5 * x))


def _esig(x):
    """Relative error of sigma(x): the exponent's rounding (of the product with log2 e, and of that
    constant), the exponential, the sum and the reciprocal."""
    return (8 + 1.3 * np.abs(x)) * U


def scan(u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, softplus=True, h0=None, dhT=None,
         dy=None, lens=None, seg=0, nseg=1, tiles=1, wrong=None):
    """(values, bounds) of y, hT and every gradient.  seg, nseg: tokens of a segment and segments
    where the sequence is cut; tiles: channel tiles of a group.  wrong: a planted mistake."""
    B, T, D = u.shape
    G, N = Bm.shape[2:]
    grp = np.arange(D) // (D // G)
    Ds = np.zeros(D) if Dskip is None else Dskip
    pre = dt + (0 if dt_bias is None else dt_bias)
    epre = 0 if dt_bias is None else U * np.abs(pre)
    if softplus:
        delta, dsp = np.logaddexp(pre, 0), _sig(pre)
        edl = (16 + 1.3 * np.abs(pre)) * U * delta + dsp * epre
        edsp = dsp * _esig(pre) + dsp * (1 - dsp) * epre
    else:
        delta, dsp, edl, edsp = pre, np.ones_like(pre), epre + 0 * pre, 0 * pre
    if wrong == "softplus":  # off where steps are small, as log(1 + e) is
        delta = np.where(pre < -4, delta * (1 + 1e-4), delta)
    if wrong == "rates":
        A = A * (1 + 1e-4)
    if wrong == "inputs":  # held in 16 bits
        u = u * (1 + 2.0 ** -9)
    if z is None:
        gate, eg = np.ones_like(pre), 0 * pre
    else:
        sz = _sig(z)
        gate = z * sz
        eg = (_esig(z) + 2 * U) * np.abs(gate)
        dgate = sz + gate * (1 - sz)
        edg = 2 * (_esig(z) + 3 * U) * (sz + np.abs(gate))
    val = {"y": np.zeros((B, T, D)), "hT": np.zeros((B, D, N)), "du": np.zeros((B, T, D)),
           "ddt": np.zeros((B, T, D)), "dA": np.zeros((D, N)), "dB": np.zeros((B, T, G, N)),
           "dC": np.zeros((B, T, G, N)), "dDskip": np.zeros(D), "ddt_bias": np.zeros(D),
           "dh0": np.zeros((B, D, N))}
    if z is not None:
        val["dz"] = np.zeros((B, T, D))
    err = {k: np.zeros_like(v) for k, v in val.items()}
    # roundings on the way through a parameter's sum: 256 tokens (their group), the groups, the
    # block's rows, the sequences' and segments' partials
    rows = B * nseg + T // 256 + 3
    cA, cP = min(T, 256) + rows, 64 + rows
    absA = {k: np.zeros_like(val[k]) for k in ("dA", "dDskip", "ddt_bias")}
    per = D // G

    def by_group(x):  # sums over a group's channels
        return x.reshape(G, per, N).sum(1)

    for b in range(B):
        n = T if lens is None else int(min(max(lens[b], 0), T))
        h = np.zeros((D, N)) if h0 is None else h0[b]
        eh = np.zeros((D, N))
        keep = []
        for t in range(n):
            d, ed, Bt, Ct = delta[b, t, :, None], edl[b, t, :, None], Bm[b, t][grp], Cm[b, t][grp]
            x = d * A
            a = np.exp(x)
            if wrong == "fold" and t % 64 == 0 and t:
                a = a * (1 + 1e-4)
            ra = EX + (2.3 + (seg if nseg > 1 else 0)) * U * np.abs(x) + np.abs(A) * ed
            w = (delta[b, t] * u[b, t])[:, None]
            ew = np.abs(u[b, t])[:, None] * ed + U * np.abs(w)
            keep.append((h, eh, a, ra, w, ew))
            ah = a * h
            eh = a * eh + ra * np.abs(ah) + np.abs(Bt) * ew + U * np.abs(w * Bt)
            h = ah + w * Bt
            eh = eh + U * np.abs(h)
            raw = (h * Ct).sum(1) + Ds * u[b, t]
            eraw = (np.abs(Ct) * eh).sum(1) + 12 * U * np.abs(h * Ct).sum(1) + \
                U * (np.abs(Ds * u[b, t]) + np.abs(raw))
            val["y"][b, t] = raw * gate[b, t]
            err["y"][b, t] = np.abs(gate[b, t]) * eraw + np.abs(raw) * (eg[b, t] + U * np.abs(gate[b, t]))
            if z is not None:
                val["dz"][b, t] = dy[b, t] * raw * dgate[b, t]
                err["dz"][b, t] = np.abs(dy[b, t]) * (np.abs(dgate[b, t]) * eraw + np.abs(raw) * edg[b, t]) + \
                    3 * U * np.abs(val["dz"][b, t])
        val["hT"][b], err["hT"][b] = h, eh
        g = np.zeros((D, N)) if dhT is None else dhT[b]
        e_g = np.zeros((D, N))
        hn, ehn = h, eh
        for t in range(n - 1, -1, -1):
            h, eh, a, ra, w, ew = keep[t]
            Bt, Ct, ut = Bm[b, t][grp], Cm[b, t][grp], u[b, t]
            e = dy[b, t] * gate[b, t]
            ee = np.abs(dy[b, t]) * eg[b, t] + U * np.abs(e)
            g = g + e[:, None] * Ct
            e_g = e_g + np.abs(Ct) * ee[:, None] + U * np.abs(g)
            c = e[:, None] * hn
            val["dC"][b, t] = by_group(c)
            err["dC"][b, t] = by_group(ehn * np.abs(e)[:, None] + np.abs(hn) * ee[:, None] +
                                       (20 + tiles) * U * np.abs(c))
            c = g * w
            val["dB"][b, t] = by_group(c)
            err["dB"][b, t] = by_group(e_g * np.abs(w) + np.abs(g) * ew + (20 + tiles) * U * np.abs(c))
            gB = (g * Bt).sum(1)
            egB = (e_g * np.abs(Bt) + 12 * U * np.abs(g * Bt)).sum(1)
            ga, ega = g * a, e_g * a + np.abs(g * a) * (ra + U)
            p = ga * h
            ep = np.abs(ga) * eh + ega * np.abs(h) + U * np.abs(p)
            d, ed = delta[b, t], edl[b, t]
            val["dA"] += p * d[:, None]
            absA["dA"] += np.abs(p * d[:, None])
            err["dA"] += ep * d[:, None] + np.abs(p) * ed[:, None]
            pA = (p * A).sum(1)
            epA = (ep * np.abs(A) + 14 * U * np.abs(p * A)).sum(1)
            s = ut * gB + pA
            es = np.abs(ut) * egB + epA + 2 * U * (np.abs(ut * gB) + np.abs(pA))
            dd = s * (dsp[b, t] if wrong != "slope" else dsp[b, t] * (1 + 1e-5))
            edd = es * dsp[b, t] + np.abs(s) * edsp[b, t] + 2 * U * np.abs(dd)
            val["ddt"][b, t], err["ddt"][b, t] = dd, edd
            val["ddt_bias"] += dd
            absA["ddt_bias"] += np.abs(dd)
            err["ddt_bias"] += edd
            val["du"][b, t] = d * gB + Ds * e
            err["du"][b, t] = ed * np.abs(gB) + np.abs(d) * egB + np.abs(Ds) * ee + \
                2 * U * (np.abs(d * gB) + np.abs(Ds * e))
            val["dDskip"] += e * ut
            absA["dDskip"] += np.abs(e * ut)
            err["dDskip"] += ee * np.abs(ut)
            g, e_g, hn, ehn = ga, ega, h, eh
            if wrong == "lost" and t % 16 == 0:  # the gradient carried over a tile
                g = g * (1 + 1e-4)
        val["dh0"][b], err["dh0"][b] = g, e_g
    for k, cnt in (("dA", cA), ("dDskip", cP), ("ddt_bias", cP)):
        err[k] += cnt * U * absA[k]
    return val, {k: 1.05 * v for k, v in err.items()}
