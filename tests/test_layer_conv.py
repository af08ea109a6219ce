"""The short causal convolution: forward, gradients, generation step, padded
batches, strided rows, histories; against the definition in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import gated_linear_sliding_chunked_b200 as L
from gated_linear_sliding_chunked_b200 import build as lbuild
from layer_ref import check, conv, np64

FAKE = 0x7F0000000000  # never dereferenced: validation fails first


def problem(seed, dtype, B, T, D, K, *, lens=None, strided=False, bias=True, hist=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    c = dict(x=r(B, T, D).to(dtype), w=r(D, K) / np.sqrt(K), dy=r(B, T, D).to(dtype),
             bias=r(D) * 0.5 if bias else None,
             x0=r(B, K - 1, D).to(dtype) if hist else None,
             dxT=r(B, K - 1, D).to(dtype) if hist else None,
             lens=None if lens is None else torch.tensor(lens))
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    if strided:  # a slice of wider rows, in a longer buffer, NaN all around
        big = torch.full((B, T + 3, 2 * D + 8), float("nan"), dtype=dtype, device="cuda")
        big[:, 2:T + 2, 8:D + 8] = d["x"]
        d["x"] = big[:, 2:T + 2, 8:D + 8]
    if lens is not None:  # what stands behind a sequence's end is not read
        for b, n in enumerate(lens):
            d["x"][b, max(n, 0):] = float("nan")
            d["dy"][b, max(n, 0):] = float("nan")
    return c, d


CASES = [  # dtype, B, T, D, K, lens, strided, bias, hist, silu
    (torch.bfloat16, 2, 37, 64, 4, None, False, True, True, True),
    (torch.bfloat16, 1, 1, 8, 4, None, False, True, False, True),
    (torch.bfloat16, 3, 100, 72, 2, [100, 0, 1], False, True, True, True),
    (torch.bfloat16, 2, 65, 40, 3, [2, 64], True, False, True, False),
    (torch.bfloat16, 1, 50, 13, 4, None, True, True, True, True),
    (torch.bfloat16, 2, 300, 128, 8, [299, 7], False, True, True, True),
    (torch.bfloat16, 2, 90, 84, 4, [90, 31], True, True, True, True),  # 8-byte vectors only
    (torch.bfloat16, 1, 33, 84, 8, None, False, True, True, True),
    (torch.bfloat16, 1, 2100, 264, 4, None, False, True, False, True),
    (torch.float32, 2, 37, 20, 4, None, False, True, True, True),
    (torch.float32, 2, 5, 1, 1, None, False, True, False, True),
    (torch.float32, 4, 33, 101, 3, [33, 32, 0, 2], True, True, True, True),
    (torch.float32, 1, 600, 36, 4, [-5], False, True, True, True),
    (torch.float32, 1, 600, 36, 6, [1000], False, False, True, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,T,D,K,lens,strided,bias,hist,silu", CASES)
def test_conv_matches_definition(dtype, B, T, D, K, lens, strided, bias, hist, silu):
    c, d = problem(T + D, dtype, B, T, D, K, lens=lens, strided=strided, bias=bias, hist=hist)
    y, xT = L.conv_fwd(d["x"], d["w"], d["bias"], d["x0"], silu=silu, lens=d["lens"],
                       want_xT=True)
    got = L.conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["x0"], d["dxT"], silu=silu,
                     lens=d["lens"], want_dx0=True)
    a = {k: np64(v) for k, v in c.items() if k != "lens"}
    ref, maj = (conv(**a, lens=lens, act=silu, absval=v) for v in (False, True))
    # K products and sums, the bias, the activation and its derivative
    k = 2 * K + 24
    check("y", y, ref["y"], maj["y"], k, dtype)
    assert np.array_equal(np64(xT), ref["xT"])
    check("dx", got["dx"], ref["dx"], maj["dx"], 2 * k, dtype)
    check("dx0", got["dx0"], ref["dx0"], maj["dx0"], 2 * k, dtype)
    # sums over every token: at most 64 in a run, 4 runs, then rows of partials
    n = 2 * k + B * T
    check("dw", got["dw"], ref["dw"], maj["dw"], n, torch.float32)
    if bias:
        check("dbias", got["dbias"], ref["dbias"], maj["dbias"], n, torch.float32)
    else:
        assert got["dbias"] is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,K", [(torch.bfloat16, 64, 4), (torch.bfloat16, 7, 2),
                                       (torch.float32, 36, 3), (torch.float32, 8, 1)])
def test_prompt_then_steps_is_the_whole_sequence(dtype, D, K):
    """A prompt in two pieces and a padded batch, then single tokens from the
    history it leaves, give the bits of one pass over everything."""
    B, T = 3, 41
    _, d = problem(5, dtype, B, T, D, K, hist=False)
    whole, xT = L.conv_fwd(d["x"], d["w"], d["bias"], want_xT=True)
    y1, h = L.conv_fwd(d["x"][:, :17], d["w"], d["bias"], want_xT=True)
    y2, h = L.conv_fwd(d["x"][:, 17:30], d["w"], d["bias"], h, want_xT=True)
    assert torch.equal(torch.cat([y1, y2], 1), whole[:, :30])
    for t in range(30, T):
        y = L.conv_step(h, d["x"][:, t], d["w"], d["bias"])
        assert torch.equal(y, whole[:, t]), t
    assert torch.equal(h, xT)
    # a padded batch of prompts of 0, 1 and 30 tokens
    n = [0, 1, 30]
    _, h = L.conv_fwd(d["x"], d["w"], d["bias"], lens=torch.tensor(n).cuda(), want_xT=True)
    y = L.conv_step(h, torch.stack([d["x"][b, n[b]] for b in range(B)]), d["w"], d["bias"])
    for b in range(B):
        assert torch.equal(y[b], whole[b, n[b]])


@pytest.mark.gpu
def test_empty_problems():
    z = dict(dtype=torch.float32, device="cuda")
    w = torch.ones(4, 3, **z)
    for B, T in ((0, 5), (2, 0)):
        y, xT = L.conv_fwd(torch.zeros(B, T, 4, **z), w, want_xT=True)
        assert y.shape == (B, T, 4) and xT.shape == (B, 2, 4)
        assert not xT.any()
        g = L.conv_bwd(torch.zeros(B, T, 4, **z), w, torch.zeros(B, T, 4, **z), w[:, 0].contiguous(),
                       dxT=torch.ones(B, 2, 4, **z), want_dx0=True)
        assert not g["dw"].any() and not g["dbias"].any()
        assert (g["dx0"] == 1).all()  # an empty sequence hands its history on


@pytest.mark.gpu
def test_one_sequence_shared_by_the_batch_and_another_stream():
    """An expanded batch reads one sequence's rows; work goes to the given
    stream; outputs are the same bits from run to run."""
    _, d = problem(9, torch.bfloat16, 1, 70, 48, 4, hist=False)
    x = d["x"].expand(3, -1, -1)
    ref, _ = L.conv_fwd(d["x"], d["w"], d["bias"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = L.conv_fwd(x, d["w"], d["bias"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(y[b], ref[0]) for b in range(3))
    dy = d["dy"].expand(3, -1, -1).contiguous()
    a, b = (L.conv_bwd(x, d["w"], dy, d["bias"]) for _ in range(2))
    assert torch.equal(a["dw"], b["dw"]) and torch.equal(a["dx"][2], b["dx"][0])


@pytest.mark.parametrize("K,act", [(1, True), (3, True), (4, False)])
def test_gradient_formula_matches_differences(K, act):
    r = np.random.default_rng(K)
    B, T, D = 2, 6, 3
    a = dict(x=r.normal(size=(B, T, D)), w=r.normal(size=(D, K)), bias=r.normal(size=D),
             x0=r.normal(size=(B, K - 1, D)))
    dy, dxT, lens = r.normal(size=(B, T, D)), r.normal(size=(B, K - 1, D)), [6, 2]
    f = lambda **q: (lambda o: (o["y"] * dy).sum() + (o["xT"] * dxT).sum())(
        conv(**{**a, **q}, lens=lens, act=act))
    g = conv(**a, lens=lens, act=act, dy=dy, dxT=dxT)
    for name, grad in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("x0", "dx0")):
        v = r.normal(size=a[name].shape)
        h = 1e-5
        diff = (f(**{name: a[name] + h * v}) - f(**{name: a[name] - h * v})) / (2 * h)
        assert abs(diff - (g[grad] * v).sum()) <= 1e-7 * (1 + abs(diff)), name


# ---- refusals (no device is touched) ----------------------------------------
@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return L.load()


def _fwd(lib, ptrs=(), **kw):
    base = dict(B=2, T=8, D=16, K=4, io=L.LZ_BF16, silu=1, ld=0, bs=0)
    base.update(kw)
    ld, bs = base.pop("ld"), base.pop("bs")
    d = L.LzConvDims(*base.values(), L.LzRows(ld, bs))
    p = dict(x=FAKE, w=FAKE + 4096, bias=None, x0=None, lens=None, y=FAKE + 8192, xT=None)
    p.update(ptrs)
    return lib.lz_conv_fwd(ctypes.byref(d), *p.values(), 0), d


@pytest.mark.parametrize("kw,status", [
    (dict(K=0), L.LZ_ERR_UNSUPPORTED), (dict(K=9), L.LZ_ERR_UNSUPPORTED),
    (dict(io=7), L.LZ_ERR_UNSUPPORTED), (dict(T=-1), L.LZ_ERR_INVALID_ARG),
    (dict(silu=2), L.LZ_ERR_INVALID_ARG), (dict(ld=-16), L.LZ_ERR_INVALID_ARG),
    (dict(B=70000), L.LZ_ERR_UNSUPPORTED), (dict(T=1 << 24), L.LZ_ERR_UNSUPPORTED)])
def test_bad_dims_rejected(lib, kw, status):
    assert _fwd(lib, **kw)[0] == status and lib.lz_last_error()
    assert L.lz_layer_workspace_bytes(_fwd(lib, **kw)[1], L.LZ_WS_CONV_BWD) == 0


@pytest.mark.parametrize("ptrs", [dict(x=None), dict(w=None), dict(y=None), dict(y=FAKE),
                                  dict(w=FAKE + 4), dict(x=FAKE + 1), dict(lens=FAKE + 4),
                                  dict(x0=FAKE + 8, xT=FAKE + 8)])
def test_bad_pointers_rejected(lib, ptrs):
    assert _fwd(lib, ptrs)[0] == L.LZ_ERR_INVALID_ARG and lib.lz_last_error()


def test_backward_and_step_refusals(lib):
    d = _fwd(lib, dict(x=None))[1]
    need = L.lz_layer_workspace_bytes(d, L.LZ_WS_CONV_BWD)
    assert need > 0
    p = [FAKE + 4096 * i for i in range(12)]
    f = lambda q, n: lib.lz_conv_bwd(ctypes.byref(d), *q, n, 0)
    assert f(p, need - 1) == L.LZ_ERR_INVALID_ARG and b"too small" in lib.lz_last_error()
    assert f(p[:11] + [None], need) == L.LZ_ERR_INVALID_ARG
    assert f(p[:8] + [None] + p[9:], need) == L.LZ_ERR_INVALID_ARG  # dw
    s = lambda *q: lib.lz_conv_step(ctypes.byref(d), *q, 0)
    assert s(None, FAKE, FAKE, None, FAKE) == L.LZ_ERR_INVALID_ARG
    assert s(FAKE, FAKE + 4096, FAKE + 8192, None, FAKE + 4096) == L.LZ_ERR_INVALID_ARG


def test_helper_refusals():
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 3)
    with pytest.raises(ValueError, match="CUDA device"):
        L.conv_fwd(x, w)
    with pytest.raises(ValueError, match="w must be"):
        L.conv_fwd(x, w.double())
    with pytest.raises(ValueError, match="lens"):
        L.conv_fwd(x, w, lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="may be strided"):
        L.conv_fwd(torch.zeros(2, 8, 5).transpose(1, 2), w)
    with pytest.raises(ValueError, match="dy"):
        L.conv_bwd(x, w, torch.zeros(2, 8, 5).transpose(1, 2))
    with pytest.raises(TypeError):
        L.conv_fwd(x.half(), w)
