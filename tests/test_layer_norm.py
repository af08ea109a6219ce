"""The block norms with gate, residual and scale: forward and gradients, rows
and attention heads, groups of every kind, odd widths; against the definition
in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import gated_linear_sliding_chunked_b200 as L
from gated_linear_sliding_chunked_b200 import build as lbuild
from layer_ref import check, norm, np64

FAKE = 0x7F0000000000
F, BF = torch.float32, torch.bfloat16


def problem(seed, dtype, B, T, D, G, parts, *, heads=False, strided=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    o = r(B, G, T, D // G) if heads else r(B, T, D)
    c = dict(o=o.to(dtype))
    for n in parts:
        c[n] = r(D) if n in ("w", "s", "w2") else r(B, T, D).to(dtype)
    d = {k: v.cuda() for k, v in c.items()}
    if strided:
        for n in ("o", "z", "r"):
            if n in d and not (heads and n == "o"):
                big = torch.full((B, T + 1, D + 24), float("nan"), dtype=dtype, device="cuda")
                big[:, 1:, 16:D + 16] = d[n]
                d[n] = big[:, 1:, 16:D + 16]
    if heads:
        c["o"] = c["o"].transpose(1, 2).reshape(B, T, D)
    return c, d


ALL = ("w", "z", "s", "r", "w2")
CASES = [  # dtype, B, T, D, G, parts, heads, strided
    (BF, 2, 5, 256, 1, ALL, False, False),
    (BF, 2, 37, 1024, 1, ALL, False, True),
    (BF, 1, 3, 64, 1, ("w",), False, False),
    (BF, 3, 11, 512, 4, ALL, True, False),
    (BF, 2, 70, 1280, 10, ("w", "z"), True, False),
    (BF, 1, 9, 768, 3, ALL, False, True),       # groups of 256: 32 lanes
    (BF, 1, 9, 1536, 3, ALL, False, False),     # groups of 512: shared memory
    (BF, 2, 7, 96, 4, ("w", "z", "r"), True, False),  # groups of 24
    (BF, 1, 4, 333, 1, ALL, False, False),
    (BF, 1, 4, 1001, 7, ALL, False, True),
    (BF, 1, 3, 30, 6, ALL, True, False),
    (BF, 2, 3, 4096, 1, ("r", "s", "w2"), False, False),  # no first norm
    (BF, 1, 2, 10240, 1, ALL, False, False),
    (BF, 1, 2, 16384, 128, ALL, False, False),
    (F, 2, 5, 128, 1, ALL, False, False),
    (F, 1, 300, 40, 5, ALL, True, False),
    (F, 1, 3, 2052, 1, ALL, False, True),
    (F, 1, 3, 1, 1, ("w", "z"), False, False),
    (F, 2, 2, 9001, 1, ALL, False, False),
    (F, 1, 700, 72, 1, ("z", "s"), False, False),
    (F, 1, 2, 16384, 2, ("w", "w2"), False, False),
    # rows on parts of a warp, the last of them past the end; rows that the same lanes come back to
    (BF, 3, 67, 64, 1, ALL, False, False),
    (BF, 2, 37, 128, 2, ALL, True, False),
    (F, 2, 45, 64, 2, ALL, False, False),       # the groups ask for 8 lanes, the row for 4
    (BF, 1, 131, 200, 1, ALL, False, True),
    (F, 2, 21, 100, 1, ALL, False, False),
    (BF, 1, 20011, 64, 1, ALL, False, False),
    (BF, 4, 33, 250, 1, ALL, False, False),
    (F, 2, 19, 50, 2, ALL, False, True),
    (BF, 1, 3, 2501, 1, ALL, False, False),
    (BF, 1, 2, 5001, 3, ALL, False, False),
    (BF, 2, 301, 8192, 1, ALL, False, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,T,D,G,parts,heads,strided", CASES)
def test_norm_matches_definition(dtype, B, T, D, G, parts, heads, strided):
    c, d = problem(B + T + D, dtype, B, T, D, G, parts, heads=heads, strided=strided)
    eps = 1e-5
    out, n = L.block_norm_fwd(**d, groups=G, eps=eps)
    a = {k: np64(v) for k, v in c.items()}
    ref, maj = (norm(**a, groups=G, eps=eps, absval=v) for v in (False, True))
    # the mean of D squares (half of its error in the root), then a few products
    k = D / 2 + 24
    check("out", out, ref["out"], maj["out"], k, dtype)
    stored = np64(out)
    g = torch.Generator().manual_seed(1)
    dout = torch.randn(B, T, D, generator=g).to(dtype)
    dn = torch.randn(B, T, D, generator=g).to(dtype) if "w2" in parts else None
    a["r"] = a.get("r")
    kw = dict(a, groups=G, eps=eps, out=stored, dout=np64(dout), dn=np64(dn))
    ref, maj = (norm(**kw, absval=v) for v in (False, True))
    if "w2" in parts:
        check("n", n, ref["n"], maj["n"], k, dtype)
    else:
        assert n is None
    d.pop("r", None)
    got = L.block_norm_bwd(**d, out=out, dout=dout.cuda(), dn=None if dn is None else dn.cuda(),
                           groups=G, eps=eps, want_dr=True)
    if heads:
        got["do"] = got["do"].transpose(1, 2).reshape(B, T, D)
    k = 4 * k
    check("dr", got["dr"], ref["dr"], maj["dr"], k, dtype)
    check("do", got["do"], ref["do"], maj["do"], k, dtype)
    for name, on in (("dz", "z"), ("dw", "w"), ("ds", "s"), ("dw2", "w2")):
        if on in parts:
            t = dtype if name == "dz" else F
            check(name, got[name], ref[name], maj[name], k + (0 if name == "dz" else B * T), t)
        else:
            assert got[name] is None


@pytest.mark.gpu
def test_one_gradient_alone_and_same_bits():
    c, d = problem(2, BF, 2, 300, 768, 1, ALL)
    out, n = L.block_norm_fwd(**d)
    d.pop("r")
    dn = torch.randn(2, 300, 768, device="cuda").bfloat16()
    a, b = (L.block_norm_bwd(**d, out=out, dn=dn) for _ in range(2))
    assert a["dr"] is None and all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)
    zero = torch.zeros_like(dn)
    e = L.block_norm_bwd(**d, out=out, dn=dn, dout=zero)
    assert all(torch.equal(a[k], e[k]) for k in a if a[k] is not None)


@pytest.mark.gpu
def test_zero_and_large_rows():
    """A row of zeros stays zero (eps in the root); rows near the largest bf16
    would overflow their squares in 32 bits and give zeros, as x / inf does:
    below 1e18 they are exact."""
    o = torch.zeros(1, 3, 256, dtype=BF, device="cuda")
    o[0, 1] = 1e18
    o[0, 2] = 1e-30
    w = torch.ones(256, device="cuda")
    out, _ = L.block_norm_fwd(o, w=w)
    assert not out[0, 0].any() and (out[0, 1] == 1).all()
    assert torch.isfinite(out).all()
    g = L.block_norm_bwd(o, w=w, dout=torch.ones_like(o))
    assert all(torch.isfinite(g[k]).all() for k in ("do", "dw"))


@pytest.mark.gpu
def test_empty_problems():
    for B, T in ((0, 4), (2, 0)):
        o, w = torch.zeros(B, T, 64, device="cuda"), torch.ones(64, device="cuda")
        out, n = L.block_norm_fwd(o, w=w, w2=w)
        assert out.shape == n.shape == (B, T, 64)
        g = L.block_norm_bwd(o, w=w, w2=w, out=out, dout=o, dn=o)
        assert not g["dw"].any() and not g["dw2"].any()


@pytest.mark.parametrize("parts,G", [(ALL, 2), (("r", "s", "w2"), 1), (("w", "z"), 3)])
def test_gradient_formula_matches_differences(parts, G):
    r = np.random.default_rng(5)
    B, T, D = 2, 3, 6
    a = dict(o=r.normal(size=(B, T, D)))
    a.update({n: r.normal(size=D if n in ("w", "s", "w2") else (B, T, D)) for n in parts})
    dout, dn = r.normal(size=(B, T, D)), r.normal(size=(B, T, D)) if "w2" in parts else None

    def f(**q):
        v = norm(**{**a, **q}, groups=G)
        return (v["out"] * dout).sum() + ((v["n"] * dn).sum() if dn is not None else 0)

    g = norm(**a, groups=G, dout=dout, dn=dn)
    grads = dict(o="do", w="dw", z="dz", s="ds", r="dr", w2="dw2")
    for name in a:
        v = r.normal(size=a[name].shape)
        h = 1e-5
        diff = (f(**{name: a[name] + h * v}) - f(**{name: a[name] - h * v})) / (2 * h)
        assert abs(diff - (g[grads[name]] * v).sum()) <= 1e-6 * (1 + abs(diff)), name


# ---- refusals (no device is touched) ----------------------------------------
@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return L.load()


def _dims(**kw):
    base = dict(B=2, T=4, D=64, G=2, heads=0, io=L.LZ_BF16, eps=1e-5)
    base.update(kw)
    return L.LzNormDims(*base.values())


def _fwd(lib, d, **ptrs):
    p = {n: FAKE + 4096 * i for i, n in enumerate(("o", "w", "z", "s", "r", "w2", "out", "n"))}
    p.update(ptrs)
    return lib.lz_block_norm_fwd(ctypes.byref(d), *p.values(), 0)


@pytest.mark.parametrize("kw,status", [
    (dict(G=5), L.LZ_ERR_INVALID_ARG), (dict(G=0), L.LZ_ERR_INVALID_ARG),
    (dict(D=16448), L.LZ_ERR_UNSUPPORTED), (dict(io=3), L.LZ_ERR_UNSUPPORTED),
    (dict(heads=2), L.LZ_ERR_INVALID_ARG), (dict(eps=0.0), L.LZ_ERR_INVALID_ARG),
    (dict(eps=float("nan")), L.LZ_ERR_INVALID_ARG), (dict(T=-1), L.LZ_ERR_INVALID_ARG)])
def test_bad_dims_rejected(lib, kw, status):
    assert _fwd(lib, _dims(**kw)) == status and lib.lz_last_error()
    assert L.lz_layer_workspace_bytes(_dims(**kw), L.LZ_WS_NORM_BWD) == 0


@pytest.mark.parametrize("ptrs", [dict(o=None), dict(out=None), dict(n=None), dict(out=FAKE),
                                  dict(w=FAKE + 4), dict(z=FAKE + 1), dict(n=FAKE + 4096 * 6)])
def test_bad_pointers_rejected(lib, ptrs):
    assert _fwd(lib, _dims(), **ptrs) == L.LZ_ERR_INVALID_ARG and lib.lz_last_error()


def test_backward_refusals(lib):
    d = _dims()
    need = L.lz_layer_workspace_bytes(d, L.LZ_WS_NORM_BWD)
    names = ("o", "w", "z", "s", "w2", "out", "dout", "dn", "do", "dz", "dr", "dw", "ds", "dw2", "ws")
    base = {n: FAKE + 4096 * i for i, n in enumerate(names)}
    bwd = lambda n=need, **q: lib.lz_block_norm_bwd(ctypes.byref(d), *{**base, **q}.values(), n, 0)
    for bad in (dict(dout=None, dn=None), dict(out=None), dict(z=None), dict(w=None), dict(s=None),
                dict(w2=None), dict(do=None), dict(ws=None), dict(dr=base["dout"])):
        assert bwd(**bad) == L.LZ_ERR_INVALID_ARG, bad
    assert bwd(n=need - 1) == L.LZ_ERR_INVALID_ARG and b"too small" in lib.lz_last_error()


def test_helper_refusals():
    o, w = torch.zeros(2, 3, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA device"):
        L.block_norm_fwd(o, w=w)
    with pytest.raises(ValueError, match="groups"):
        L.block_norm_fwd(torch.zeros(2, 4, 3, 8), w=torch.zeros(32), groups=2)
    with pytest.raises(ValueError, match="w must be"):
        L.block_norm_fwd(o, w=torch.zeros(7))
    with pytest.raises(ValueError, match="dout or dn"):
        L.block_norm_bwd(o, w=w)
    with pytest.raises(ValueError, match="needs out"):
        L.block_norm_bwd(o, w=w, w2=w, dn=o)
