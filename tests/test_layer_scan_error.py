"""The scan's outputs within what 32-bit arithmetic may be off by, by a bound that every element
carries along (scan_error.py); the bound itself against planted mistakes; and sequences long enough
that every buffer of the kernels' pipelines comes into use again."""
import numpy as np
import pytest
import torch

import gated_linear_sliding_chunked_b200 as L
import scan_error
from layer_ref import HALF, np64
from test_layer_scan import BF, CASES, F, problem

SMS = 148


def _plan(B, T, D, G, N):
    """Tokens of a segment, segments and channel tiles, as the library cuts a call."""
    n, per = 4, D // G
    while n < N:
        n *= 2
    tiles = -(-per // (512 // n))
    base = tiles * G * B
    k = min(32, 2 * SMS // base) if base * 3 <= 2 * SMS else 1
    if k == 1:
        return T, 1, tiles
    seg = max(64, -(-(-(-T // k)) // 32) * 32)
    return seg, max(1, -(-T // seg)), tiles


def _check(c, d, lens, softplus, hold=None):
    B, T, D = c["u"].shape
    G, N = c["Bm"].shape[2:]
    dy, dhT = d.pop("dy"), d.pop("dhT", None)
    a = [d.pop(k) for k in ("u", "dt", "A", "Bm", "Cm")]
    y, hT, states = L.scan_fwd(*a, **d, softplus=softplus, want_hT=True, want_states=True)
    got = L.scan_bwd(*a, dy, **d, softplus=softplus, dhT=dhT, want_dh0=True, states=states)
    got.update(y=y, hT=hT)
    seg, nseg, tiles = _plan(B, T, D, G, N)
    val, err = scan_error.scan(**{k: np64(v) for k, v in c.items()}, softplus=softplus, lens=lens,
                               seg=seg, nseg=nseg, tiles=tiles)
    worst = {}
    for k, ref in val.items():
        if got[k] is None:
            continue
        x = np64(got[k])
        assert np.isfinite(x).all(), k
        tol = HALF[got[k].dtype] * np.abs(ref) * (1 + 2.0 ** -7) + err[k] + 1e-36
        worst[k] = float((np.abs(x - ref) / tol).max()) if ref.size else 0.0
    assert max(worst.values()) <= 1, worst


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,T,D,G,N,z,h0,skip,lens,strided,softplus", CASES)
def test_scan_within_its_roundings(dtype, B, T, D, G, N, z, h0, skip, lens, strided, softplus):
    c, d = problem(T + D + N, dtype, B, T, D, G, N, z=z, h0=h0, skip=skip, lens=lens,
                   strided=strided, softplus=softplus)
    _check(c, d, lens, softplus)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [4, 8, 12, 16, 24, 32, 48, 64])
def test_slow_decays_over_segments(N):
    """Steps of some 0.004: a state keeps a third of itself over a segment of 64 tokens, so that
    every segment's end reaches the ones behind."""
    c, d = problem(N, F, 2, 300, 48, 2, N, lens=[300, 211])
    d["dt_bias"] -= 3
    c["dt_bias"] -= 3
    _check(c, d, [300, 211], True)


STEADY = [  # dtype, B, T, D, G, N: pipelines of at least four tiles
    # blocks of seven scan and seven elementwise warps
    (BF, 1, 139, 4800, 1, 16), (F, 1, 130, 4800, 2, 16), (BF, 1, 139, 2400, 1, 32), (F, 1, 139, 2400, 1, 32),
    (BF, 1, 139, 1200, 1, 64), (F, 1, 133, 1200, 1, 64),
    # blocks with an SM to themselves: four scan warps, eight elementwise ones
    (BF, 1, 139, 3200, 1, 16), (F, 1, 139, 3200, 1, 16), (BF, 1, 139, 1600, 1, 32), (F, 1, 130, 1600, 2, 32),
    (BF, 1, 75, 6400, 1, 8), (F, 1, 75, 6400, 1, 8), (BF, 1, 43, 12800, 1, 4), (F, 1, 43, 12800, 1, 4),
    # two blocks an SM
    (BF, 3, 139, 1600, 1, 32), (F, 2, 75, 6400, 1, 8), (F, 2, 139, 800, 1, 64), (BF, 2, 43, 12800, 1, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,T,D,G,N", STEADY)
def test_pipelines_in_their_steady_state(dtype, B, T, D, G, N):
    assert _plan(B, T, D, G, N)[1] == 1
    c, d = problem(D + N, dtype, B, T, D, G, N, lens=[T] * (B - 1) + [T - 5])
    _check(c, d, [T] * (B - 1) + [T - 5], True)


@pytest.mark.parametrize("wrong,names", [
    ("inputs", ("y", "hT", "ddt", "dA", "dB", "dC", "dDskip", "ddt_bias", "dz")),
    ("rates", ("y", "hT", "du", "ddt", "dA", "dB", "dC", "dz", "dh0")),
    ("softplus", ("y", "hT", "du", "ddt", "dA", "dB", "dC", "dz", "dh0")),
    ("slope", ("ddt",)),
    ("fold", ("y", "hT", "du", "ddt", "dA", "dB", "dC", "dz", "dh0")),
    ("lost", ("du", "ddt", "dA", "dB", "dh0"))])
@pytest.mark.parametrize("N", [8, 16])
def test_the_bound_shows_mistakes(wrong, names, N):
    """Inputs held in 16 bits, rates, steps and carried states and gradients off by 1e-4, a
    derivative by 1e-5: each leaves the bound of a 32-bit call in every output that it reaches."""
    B, T, D, G = 2, 150, 16, 2
    r = np.random.default_rng(N).normal
    a = dict(u=r(size=(B, T, D)), dt=r(size=(B, T, D)), dy=r(size=(B, T, D)), z=r(size=(B, T, D)),
             Bm=r(size=(B, T, G, N)), Cm=r(size=(B, T, G, N)), h0=r(size=(B, D, N)), dhT=r(size=(B, D, N)),
             A=-np.exp(0.5 * r(size=(D, N))) * (1 + np.arange(N) % 5), Dskip=r(size=D), dt_bias=r(size=D) - 4.5)
    seg, nseg, tiles = _plan(B, T, D, G, N)
    val, err = scan_error.scan(**a, seg=seg, nseg=nseg, tiles=tiles)
    bad, _ = scan_error.scan(**a, seg=seg, nseg=nseg, tiles=tiles, wrong=wrong)
    for k in names:
        assert (np.abs(bad[k] - val[k]) > 2.0 ** -24 * np.abs(val[k]) * (1 + 2.0 ** -7) + err[k]).any(), k
