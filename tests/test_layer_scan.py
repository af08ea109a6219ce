"""The selective state space scan: forward, gradients, generation step, padded
batches, strided rows, groups, carried states; against the definition in 64
bits."""
import ctypes

import numpy as np
import pytest
import torch

import gated_linear_sliding_chunked_b200 as L
from gated_linear_sliding_chunked_b200 import build as lbuild
from layer_ref import check, np64, scan

FAKE = 0x7F0000000000
F, BF = torch.float32, torch.bfloat16


def problem(seed, dtype, B, T, D, G, N, *, z=True, h0=True, skip=True, lens=None, strided=False,
            softplus=True, dt_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    c = dict(u=r(B, T, D).to(dtype), dt=(dt_scale * r(B, T, D)).to(dtype),
             A=-torch.exp(0.5 * r(D, N)) * (1 + torch.arange(N) % 5),
             Bm=r(B, T, G, N).to(dtype), Cm=r(B, T, G, N).to(dtype), dy=r(B, T, D).to(dtype))
    if softplus:
        c["dt_bias"] = r(D) - 2.5
    else:
        c["dt"] = (c["dt"].abs() * 0.1).to(dtype)
    if z:
        c["z"] = r(B, T, D).to(dtype)
    if skip:
        c["Dskip"] = r(D)
    if h0:
        c["h0"], c["dhT"] = r(B, D, N), r(B, D, N)
    d = {k: v.cuda() for k, v in c.items()}
    if strided:  # u | z and dt | B | C as one projection's rows, NaN all around
        for names in (("u", "z"), ("dt", "Bm", "Cm")):
            names = [n for n in names if n in d]
            parts = [d[n].flatten(2) for n in names]
            wide = sum(p.shape[2] for p in parts)
            big = torch.full((B, T + 2, wide + 8), float("nan"), dtype=dtype, device="cuda")
            at = 8
            for n, p in zip(names, parts):
                big[:, 1:T + 1, at:at + p.shape[2]] = p
                d[n] = big[:, 1:T + 1, at:at + p.shape[2]].unflatten(2, tuple(d[n].shape[2:]))
                at += p.shape[2]
    if lens is not None:
        for n in ("u", "dt", "z", "Bm", "Cm", "dy"):
            if n in d:
                for b, e in enumerate(lens):
                    d[n][b, max(e, 0):] = float("nan")
        d["lens"] = torch.tensor(lens).cuda()
    return c, d


def refs(c, lens, softplus, **more):
    a = {k: np64(v) for k, v in c.items()}
    a.update(more)
    return (scan(**a, softplus=softplus, lens=lens, absval=v) for v in (False, True))


def roundings(c, T, softplus):
    """Roundings on the longest way through the recurrence: a few a token, the
    exponent's relative to itself (|delta A| of them for each)."""
    pre = c["dt"].float() + c.get("dt_bias", torch.zeros(1))
    delta = torch.nn.functional.softplus(pre) if softplus else pre
    top = float((delta.reshape(-1, delta.shape[-1]).amax(0) * c["A"].abs().amax(1)).max()) \
        if delta.numel() else 0.0
    return (8 * T + 64) * (1 + top)


CASES = [  # dtype, B, T, D, G, N, z, h0, skip, lens, strided, softplus
    (BF, 2, 48, 64, 1, 16, True, True, True, None, False, True),
    (BF, 1, 1, 8, 1, 16, True, False, True, None, False, True),
    (BF, 3, 100, 48, 2, 16, True, True, True, [100, 0, 1], False, True),
    (BF, 2, 257, 40, 1, 16, False, True, False, None, True, True),
    (BF, 1, 130, 72, 3, 8, True, True, True, None, True, True),
    (BF, 2, 77, 13, 1, 12, True, True, True, [77, 33], True, True),
    (BF, 2, 65, 136, 1, 4, True, False, True, None, False, True),
    (BF, 2, 150, 24, 3, 64, True, True, True, [64, 150], False, True),
    (BF, 1, 90, 32, 2, 32, False, False, True, None, False, False),
    (F, 2, 48, 64, 1, 16, True, True, True, None, False, True),
    (F, 2, 193, 20, 2, 8, True, True, True, [193, 64], False, True),
    (F, 3, 31, 7, 7, 20, True, True, False, [16, 17, 15], True, True),
    (F, 1, 300, 9, 1, 64, False, True, True, None, True, False),
    (F, 2, 16, 1, 1, 4, True, False, True, None, False, True),
    (F, 1, 513, 132, 1, 4, True, True, True, [512], False, True),
    (F, 1, 2, 300, 2, 16, True, True, True, [-3], False, True),
    (F, 4, 33, 3000, 1, 16, True, True, True, [99, 33, 32, 31], False, True),
    # as many channels as blocks of seven scan warps are taken for
    (BF, 2, 35, 4096, 1, 16, True, True, True, [35, 18], False, True),
    (F, 2, 17, 4090, 2, 16, True, False, True, None, False, True),
    (BF, 2, 33, 2040, 1, 32, False, True, True, None, True, True),
    (F, 2, 20, 1020, 2, 52, True, True, True, [20, 3], False, True),
    (BF, 2, 18, 1024, 1, 64, True, False, True, None, False, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,T,D,G,N,z,h0,skip,lens,strided,softplus", CASES)
def test_scan_matches_definition(dtype, B, T, D, G, N, z, h0, skip, lens, strided, softplus):
    c, d = problem(T + D + N, dtype, B, T, D, G, N, z=z, h0=h0, skip=skip, lens=lens,
                   strided=strided, softplus=softplus)
    dy, dhT = d.pop("dy"), d.pop("dhT", None)
    a = [d.pop(k) for k in ("u", "dt", "A", "Bm", "Cm")]
    y, hT, states = L.scan_fwd(*a, **d, softplus=softplus, want_hT=True, want_states=True)
    kw = dict(d, softplus=softplus, dhT=dhT, want_dh0=True)
    got = L.scan_bwd(*a, dy, **kw, states=states)
    ref, maj = refs(c, lens, softplus)
    k = roundings(c, T, softplus)
    check("y", y, ref["y"], maj["y"], k, dtype)
    check("hT", hT, ref["hT"], maj["hT"], k, F)
    names = ["du", "ddt", "dB", "dC"] + ["dz"] * z
    for n in names:  # dB, dC: sums over the channels
        check(n, got[n], ref[n], maj[n], 2 * k + D, dtype)
    for n in ["dA", "ddt_bias", "dh0"] + ["dDskip"] * skip:
        if n == "ddt_bias" and not softplus:
            assert got[n] is None
            continue
        check(n, got[n], ref[n], maj[n], 2 * k + B * T, F)
    # without the saved states the call walks forward itself: the same bits
    again = L.scan_bwd(*a, dy, **kw)
    for n, x in got.items():
        assert (x is None and again[n] is None) or torch.equal(x, again[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("N", [4, 8, 12, 16, 24, 32, 48, 64])
def test_every_width_of_state(dtype, N):
    """Whole vectors of channels, several tiles and segments, at every width:
    each has its own split of states over lanes and of tokens over threads."""
    test_scan_matches_definition(dtype, 2, 150, 64, 2, N, True, True, True, [150, 97], False, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,G,N", [(BF, 64, 1, 16), (BF, 9, 3, 12), (F, 40, 2, 64),
                                         (F, 5, 1, 4)])
def test_prompt_then_steps_is_the_whole_sequence(dtype, D, G, N):
    """Prompt in two pieces, then single tokens, against one pass: the state
    agrees to the recurrence's own roundings."""
    B, T = 3, 71
    c, d = problem(3, dtype, B, T, D, G, N, h0=False)
    args = lambda s: [d["u"][:, s], d["dt"][:, s], d["A"], d["Bm"][:, s], d["Cm"][:, s]]
    kw = lambda s: dict(Dskip=d["Dskip"], dt_bias=d["dt_bias"], z=d["z"][:, s])
    k = roundings(c, T, True)
    c = {n: v for n, v in c.items() if n not in ("dy",)}
    ref, maj = refs(c, None, True)
    y1, h = L.scan_fwd(*args(slice(0, 33)), **kw(slice(0, 33)), want_hT=True)
    y2, h = L.scan_fwd(*args(slice(33, 60)), **kw(slice(33, 60)), h0=h, want_hT=True)
    ys = [y1, y2] + [L.scan_step(h, *args(t), **kw(t))[:, None] for t in range(60, T)]
    check("y", torch.cat(ys, 1), ref["y"], maj["y"], k, dtype)
    check("state", h, ref["hT"], maj["hT"], k, F)


@pytest.mark.gpu
def test_padded_prompts_continue_with_steps():
    B, T, D, N = 4, 50, 24, 16
    c, d = problem(8, F, B, T, D, 1, N, h0=False)
    lens = [50, 0, 1, 32]
    a = [d[k] for k in ("u", "dt", "A", "Bm", "Cm")]
    kw = {k: d[k] for k in ("Dskip", "dt_bias", "z")}
    _, h = L.scan_fwd(*a, **kw, lens=torch.tensor(lens).cuda(), want_hT=True)
    for b, n in enumerate(lens):
        one = [x[b:b + 1, :n] if x.dim() > 2 else x for x in a]
        _, hb = L.scan_fwd(*one, Dskip=d["Dskip"], dt_bias=d["dt_bias"], z=d["z"][b:b + 1, :n],
                           want_hT=True)
        assert torch.allclose(h[b], hb[0], rtol=1e-4, atol=1e-6), b


@pytest.mark.gpu
def test_long_sequence():
    """65536 tokens of few channels (the segmented path).  Decays of at most
    1/2 a token keep what is behind out of the error: a token's error is that
    of the last few, E = a (E + eps H) + eps H <= 2 k eps max H."""
    B, T, D, N = 1, 65536, 8, 4
    g = torch.Generator().manual_seed(1)
    u, Bm, Cm = (torch.rand(B, T, *s, generator=g) + 0.5 for s in ((D,), (1, N), (1, N)))
    dt, A = torch.rand(B, T, D, generator=g) * 0.1 + 0.7, -torch.ones(D, N)
    c = dict(u=u, dt=dt, A=A, Bm=Bm, Cm=Cm)
    y, hT = L.scan_fwd(*(v.cuda() for v in c.values()), softplus=False, want_hT=True)
    ref, maj = refs(c, None, False)
    top = np.broadcast_to(maj["y"].max(), ref["y"].shape)
    check("y", y, ref["y"], top, 64, F)
    check("hT", hT, ref["hT"], np.broadcast_to(maj["hT"].max(), ref["hT"].shape), 64, F)


@pytest.mark.gpu
def test_strong_and_vanishing_decay():
    """delta A of -400 forgets everything (the state is the token's input, no
    NaN); delta near 0 (softplus of -30) keeps the state's bits."""
    B, T, D, N = 1, 40, 16, 16
    c, d = problem(4, F, B, T, D, 1, N, z=False)
    d["dt"].fill_(400.0)
    a = [d[k] for k in ("u", "dt", "A", "Bm", "Cm")]
    d["A"].clamp_(max=-1.0)
    kw = dict(h0=d["h0"], Dskip=d["Dskip"])
    y, hT = L.scan_fwd(*a, **kw, want_hT=True)
    want = 400.0 * d["u"][:, -1, :, None] * d["Bm"][:, -1]
    assert torch.allclose(hT, want, rtol=1e-6, atol=0)
    g = L.scan_bwd(*a, d["dy"], **kw, dhT=d["dhT"], want_dh0=True)
    assert all(torch.isfinite(x).all() for x in g.values() if x is not None)
    assert not g["dh0"].any()
    d["dt"].fill_(-110.0)
    y, hT = L.scan_fwd(*a, **kw, want_hT=True)
    assert torch.allclose(hT, d["h0"], rtol=1e-6, atol=1e-30)


@pytest.mark.gpu
def test_gradients_match_differences_of_the_forward():
    """Directional differences of the kernel's own forward in 32 bits."""
    B, T, D, N = 2, 33, 24, 8
    c, d = problem(6, F, B, T, D, 2, N)
    dy, dhT = d.pop("dy"), d.pop("dhT")
    g = L.scan_bwd(*(d[k] for k in ("u", "dt", "A", "Bm", "Cm")), dy,
                   **{k: d[k] for k in ("Dskip", "z", "dt_bias", "h0")}, dhT=dhT, want_dh0=True)

    def f(**q):
        v = {**d, **q}
        a = [v.pop(k) for k in ("u", "dt", "A", "Bm", "Cm")]
        y, hT = L.scan_fwd(*a, **v, want_hT=True)
        return float((y.double() * dy).sum() + (hT.double() * dhT).sum())

    gen = torch.Generator(device="cuda").manual_seed(0)
    for name, grad in (("u", "du"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"),
                       ("Dskip", "dDskip"), ("z", "dz"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        v = torch.randn(d[name].shape, generator=gen, device="cuda")
        h = 2.0 ** -8
        diff = (f(**{name: d[name] + h * v}) - f(**{name: d[name] - h * v})) / (2 * h)
        want = float((g[grad].double() * v).sum())
        # the difference's third-order term is h^2 of the scale of the slope,
        # the values' roundings 2^-24 / h of theirs: both below 1e-3 of it
        scale = float((g[grad].double().abs() * v.abs()).sum())
        assert abs(diff - want) <= 1e-3 * scale, (name, diff, want)


@pytest.mark.gpu
def test_captured_calls_replay():
    """Forward and backward in a CUDA graph, replayed on new inputs."""
    c, d = problem(7, BF, 2, 70, 64, 1, 16, h0=False)
    c2, d2 = problem(17, BF, 2, 70, 64, 1, 16, h0=False)
    names = ("u", "dt", "A", "Bm", "Cm", "dy", "Dskip", "z", "dt_bias")

    def call(v):
        kw = {k: v[k] for k in ("Dskip", "z", "dt_bias")}
        a = [v[k] for k in ("u", "dt", "A", "Bm", "Cm")]
        y, _, st = L.scan_fwd(*a, **kw, want_states=True)
        return [y] + [x for x in L.scan_bwd(*a, v["dy"], **kw, states=st).values()
                      if x is not None]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(d)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(d)
    want = call(d2)
    for n in names:
        d[n].copy_(d2[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, want))


@pytest.mark.gpu
def test_empty_problems():
    z = dict(dtype=F, device="cuda")
    A = -torch.ones(8, 4, **z)
    for B, T in ((0, 5), (2, 0)):
        u, bc, h = torch.zeros(B, T, 8, **z), torch.zeros(B, T, 4, **z), torch.ones(B, 8, 4, **z)
        y, hT, st = L.scan_fwd(u, u, A, bc, bc, h0=h, want_hT=True, want_states=True)
        assert y.shape == (B, T, 8) and torch.equal(hT, h)
        g = L.scan_bwd(u, u, A, bc, bc, u, h0=h, dhT=2 * h, states=st, want_dh0=True)
        assert torch.equal(g["dh0"], 2 * h) and not g["dA"].any()


@pytest.mark.parametrize("softplus,z", [(True, True), (False, False)])
def test_gradient_formula_matches_differences(softplus, z):
    r = np.random.default_rng(3)
    B, T, D, G, N = 2, 5, 4, 2, 3
    a = dict(u=r.normal(size=(B, T, D)), dt=r.normal(size=(B, T, D)), A=-np.exp(r.normal(size=(D, N))),
             Bm=r.normal(size=(B, T, G, N)), Cm=r.normal(size=(B, T, G, N)), Dskip=r.normal(size=D),
             dt_bias=r.normal(size=D), h0=r.normal(size=(B, D, N)))
    if z:
        a["z"] = r.normal(size=(B, T, D))
    dy, dhT, lens = r.normal(size=(B, T, D)), r.normal(size=(B, D, N)), [5, 3]
    f = lambda **q: (lambda o: (o["y"] * dy).sum() + (o["hT"] * dhT).sum())(
        scan(**{**a, **q}, softplus=softplus, lens=lens))
    g = scan(**a, softplus=softplus, lens=lens, dy=dy, dhT=dhT)
    grads = dict(u="du", dt="ddt", A="dA", Bm="dB", Cm="dC", Dskip="dDskip", dt_bias="ddt_bias",
                 h0="dh0", z="dz")
    # a value of f is off by up to 64 roundings of 2^-53 of its majorant (without
    # softplus delta may be negative, the state grows and f with it), which the
    # difference divides by h
    maj = scan(**a, softplus=softplus, lens=lens, absval=True)
    off = 64 * 2.0 ** -53 * ((maj["y"] * abs(dy)).sum() + (maj["hT"] * abs(dhT)).sum()) / 1e-5
    for name in a:
        v = r.normal(size=a[name].shape)
        h = 1e-5
        diff = (f(**{name: a[name] + h * v}) - f(**{name: a[name] - h * v})) / (2 * h)
        assert abs(diff - (g[grads[name]] * v).sum()) <= 1e-6 * (1 + abs(diff)) + off, name


# ---- refusals (no device is touched) ----------------------------------------
@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return L.load()


def _dims(**kw):
    base = dict(B=2, T=8, D=16, G=2, N=16, io=L.LZ_BF16, softplus=1)
    ld = kw.pop("ld", 0)
    base.update(kw)
    return L.LzScanDims(*base.values(), L.LzRows(ld, 0))


def _fwd(lib, d, **ptrs):
    names = ("u", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "h0", "lens", "y", "hT",
             "states", "ws")
    p = {n: FAKE + 4096 * i for i, n in enumerate(names)}
    n = ptrs.pop("n", 1 << 40)
    p.update(ptrs)
    return lib.lz_scan_fwd(ctypes.byref(d), *p.values(), n, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(N=2), L.LZ_ERR_UNSUPPORTED), (dict(N=18), L.LZ_ERR_UNSUPPORTED),
    (dict(N=68), L.LZ_ERR_UNSUPPORTED), (dict(G=3), L.LZ_ERR_INVALID_ARG),
    (dict(G=0), L.LZ_ERR_INVALID_ARG), (dict(io=5), L.LZ_ERR_UNSUPPORTED),
    (dict(softplus=3), L.LZ_ERR_INVALID_ARG), (dict(B=-1), L.LZ_ERR_INVALID_ARG),
    (dict(T=1 << 24), L.LZ_ERR_UNSUPPORTED), (dict(ld=-1), L.LZ_ERR_INVALID_ARG)])
def test_bad_dims_rejected(lib, kw, status):
    d = _dims(**kw)
    assert _fwd(lib, d) == status and lib.lz_last_error()
    assert L.lz_layer_workspace_bytes(d, L.LZ_WS_SCAN_BWD) == 0
    p = [FAKE + 4096 * i for i in range(10)]
    if "T" not in kw:
        assert lib.lz_scan_step(ctypes.byref(d), *p, 0) == status


@pytest.mark.parametrize("ptrs", [dict(u=None), dict(A=None), dict(Cm=None), dict(A=FAKE + 8),
                                  dict(y=FAKE), dict(lens=FAKE + 4), dict(dt=FAKE + 1),
                                  dict(hT=FAKE + 4096 * 8), dict(ws=FAKE + 16)])
def test_bad_pointers_rejected(lib, ptrs):
    assert _fwd(lib, _dims(), **ptrs) == L.LZ_ERR_INVALID_ARG and lib.lz_last_error()


def test_workspace_and_backward_refusals(lib):
    d = _dims(T=4096)
    need = L.lz_layer_workspace_bytes(d, L.LZ_WS_SCAN_FWD)
    assert need > 0  # few channels: segments
    assert _fwd(lib, d, n=need - 1) == L.LZ_ERR_INVALID_ARG and b"too small" in lib.lz_last_error()
    p = [FAKE + 4096 * i for i in range(23)]
    bwd = lambda q, n: lib.lz_scan_bwd(ctypes.byref(d), *q, n, 0)
    need = L.lz_layer_workspace_bytes(d, L.LZ_WS_SCAN_BWD)
    assert bwd(p, need - 1) == L.LZ_ERR_INVALID_ARG and b"too small" in lib.lz_last_error()
    assert bwd(p[:6] + [None] + p[7:], need) == L.LZ_ERR_INVALID_ARG  # dz without z
    assert bwd(p[:15] + [None] + p[16:], need) == L.LZ_ERR_INVALID_ARG  # dA
    assert bwd(p[:14] + [p[13]] + p[15:], need) == L.LZ_ERR_INVALID_ARG  # du is ddt


def test_helper_refusals():
    u, bc, A = torch.zeros(2, 5, 8), torch.zeros(2, 5, 4), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA device"):
        L.scan_fwd(u, u, A, bc, bc)
    with pytest.raises(ValueError, match="Cm"):
        L.scan_fwd(u, u, A, bc, torch.zeros(2, 5, 8))
    with pytest.raises(ValueError, match="h0"):
        L.scan_fwd(u, u, A, bc, bc, h0=torch.zeros(2, 8, 5))
    with pytest.raises(ValueError, match="dt_bias"):
        L.scan_fwd(u, u, A, bc, bc, dt_bias=torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="states"):
        L.scan_bwd(u, u, A, bc, bc, u, states=torch.zeros(3))
    with pytest.raises(ValueError, match="shared by all tokens"):
        L.scan_fwd(u, u, A, bc[:, :1].expand(-1, 5, -1), bc)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F, BF])
def test_growing_states(dtype):
    """Rates of both signs, decays up to e^2 a token: values and gradients against autograd in 64
    bits.  12 tokens, some 8 roundings of 2^-24 each and the decays' 2^-22, none of which cancels
    more than the sums do: 12 (8 2^-24 + 2^-22) = 9e-6, and 2^-8 for what leaves in 16 bits."""
    B, T, D, N = 2, 12, 24, 8
    gen = torch.Generator().manual_seed(3)
    u, dy = (torch.randn(B, T, D, generator=gen).to(dtype) for _ in range(2))
    dt = (1 + torch.rand(B, T, D, generator=gen)).to(dtype)
    Bm, Cm = (torch.randn(B, T, N, generator=gen).to(dtype) for _ in range(2))
    A = 2 * torch.rand(D, N, generator=gen) - 1
    leaves = [t.double().requires_grad_() for t in (u, dt, A, Bm, Cm)]
    u64, dt64, A64, B64, C64 = leaves
    h, ys = torch.zeros(B, D, N, dtype=torch.float64), []
    for t in range(T):
        h = torch.exp(dt64[:, t, :, None] * A64) * h + (dt64 * u64)[:, t, :, None] * B64[:, t, None]
        ys.append((h * C64[:, t, None]).sum(-1))
    y64 = torch.stack(ys, 1)
    (y64 * dy.double()).sum().backward()
    a = [t.cuda() for t in (u, dt, A, Bm, Cm)]
    y, _ = L.scan_fwd(*a, softplus=False)
    g = L.scan_bwd(*a, dy.cuda(), softplus=False)
    got = [y, g["du"], g["ddt"], g["dA"], g["dB"], g["dC"]]
    for name, x, ref in zip(("y", "du", "ddt", "dA", "dB", "dC"), got,
                            [y64.detach()] + [t.grad for t in leaves]):
        err = float((x.double().cpu() - ref).norm() / ref.norm())
        assert err <= (9e-6 if x.dtype == F else 9e-6 + 2 ** -8), (name, err)
