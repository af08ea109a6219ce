"""The scan's decays: their mean error, which a state's memory multiplies.

With u = 0 the last state is h0 times the product of all decays, so log(hT / h0) against the exact
exponents shows the sum of the decays' relative errors (and of the products' roundings, whose mean
is zero)."""
import math

import pytest
import torch

import gated_linear_sliding_chunked_b200 as L

pytestmark = pytest.mark.gpu

D, N = 64, 16
BINADES = range(-12, -1)  # of the exponents |delta A log2 e|


def _problem(k, B):
    """Exponents of one binade, uniform in it; as many tokens as keep the state within a float."""
    g = torch.Generator().manual_seed(100 - k)
    T = min(2048, 32 * 2 ** -k)
    A = -0.5 - torch.rand(D, N, generator=g)
    dt = (1 + torch.rand(B, T, D, generator=g)) * (2.0 ** k / math.log2(math.e))
    x = dt.double().sum(1)[..., None] * A.double()
    return T, A.cuda(), dt.cuda(), x


def _mean(out, x, T):
    """Mean relative error of a decay: over the channels, states and sequences, a token."""
    return float((torch.log(out.double().cpu()) - x).mean()) / T


def _forward(T, A, dt, x):
    B = dt.shape[0]
    u, bc = torch.zeros(B, T, D, device="cuda"), torch.zeros(B, T, N, device="cuda")
    h0 = torch.ones(B, D, N, device="cuda")
    return L.scan_fwd(u, dt, A, bc, bc, softplus=False, h0=h0, want_hT=True)[1]


def _backward(T, A, dt, x):
    B = dt.shape[0]
    u, bc = torch.zeros(B, T, D, device="cuda"), torch.zeros(B, T, N, device="cuda")
    dhT = torch.ones(B, D, N, device="cuda")
    return L.scan_bwd(u, dt, A, bc, bc, u, softplus=False, dhT=dhT, want_dh0=True)["dh0"]


def _steps(T, A, dt, x):
    B = dt.shape[0]
    u, bc = torch.zeros(B, D, device="cuda"), torch.zeros(B, N, device="cuda")
    h = torch.ones(B, D, N, device="cuda")
    for t in range(T):
        L.scan_step(h, u, dt[:, t].contiguous(), A, bc, bc, softplus=False)
    return h


@pytest.mark.parametrize("run,B", [(_forward, 50), (_backward, 50), (_forward, 1), (_backward, 1),
                                   (_steps, 4)])
def test_decays_have_no_mean_error(run, B):
    """A decay just below 1 is stored to 2^-24 of itself, so one rounding is off by at most 2^-25, and
    by 0 on average.  The mean error over all binades is held to a quarter of that, 2^-27: over a
    memory of 1000 tokens it makes 7.5e-6.  So is that of a binade of slow decays (memories of 350
    tokens and more); a binade of fast ones alone is held to three times as much.  What is random,
    some 2^-24 a token, is below 2^-24 / sqrt(T D B) <= 2^-24 / 90 in the mean.

    (50 sequences' blocks fill the device and walk whole sequences; one is cut into segments.)"""
    means = {}
    for k in BINADES:
        T, A, dt, x = _problem(k, B)
        means[k] = _mean(run(T, A, dt, x), x, T)
    assert abs(sum(means.values())) / len(means) <= 2.0 ** -27
    for k, m in means.items():
        assert abs(m) <= (2.0 ** -27 if k <= -9 else 3 * 2.0 ** -27), (k, m)


def test_parameter_gradients_over_many_tokens():
    """16384 equal terms a channel, each a little above 1, so that one 32-bit sum over a thread's 1024
    of them rounds down every time (1.5e-5 of the result).  Summed over 16 tiles of tokens at a time
    the longest way through the sums has 16 + 64 + 16 + 1 roundings of 2^-24: 5.8e-6."""
    T, D, N = 16384, 800, 64  # 100 blocks: sequences are not cut
    c = 1 + 0.49 * 2.0 ** -14
    u = torch.full((1, T, D), c, device="cuda")
    bc = torch.zeros(1, T, N, device="cuda")
    A, Ds = -torch.ones(D, N, device="cuda"), torch.ones(D, device="cuda")
    dy = torch.ones(1, T, D, device="cuda")
    got = L.scan_bwd(u, torch.full_like(u, 0.1), A, bc, bc, dy, softplus=False, Dskip=Ds)["dDskip"]
    want = T * float(u[0, 0, 0].double())
    assert float((got.double() - want).abs().max()) <= 97 * 2.0 ** -24 * want
