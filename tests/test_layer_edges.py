"""Layer operators where a value overflows, a length ends or a call meets another device: against the
definitions in 64 bits."""
import numpy as np
import pytest
import torch

import gated_linear_sliding_chunked_b200 as L
from layer_ref import np64, scan


def _growing(T, dt, u_on, dy_on, h0=None, dhT=None):
    """Inputs of one sequence (8 channels, 4 states, rates of 1: one block, cut into segments of 64
    tokens) with u and dy zero outside the given tokens, the reference and the kernel's results."""
    D, N = 8, 4
    g = torch.Generator().manual_seed(T)
    pos = lambda *s: torch.rand(*s, generator=g) + 0.5
    only = lambda x, on: x * torch.zeros(T, 1).index_fill(0, torch.tensor(on), 1.0)
    c = dict(u=only(pos(1, T, D), u_on), dt=dt.expand(1, D, T).transpose(1, 2).contiguous(),
             A=torch.ones(D, N), Bm=pos(1, T, 1, N), Cm=pos(1, T, 1, N))
    dy = only(pos(1, T, D), dy_on)
    more = {k: torch.full((1, D, N), v) for k, v in (("h0", h0), ("dhT", dhT)) if v is not None}
    ref = scan(**{k: np64(v) for k, v in {**c, **more, "dy": dy}.items()}, softplus=False)
    a = [v.cuda() for v in c.values()]
    m = {k: v.cuda() for k, v in more.items()}
    y, hT = L.scan_fwd(*a, softplus=False, h0=m.get("h0"), want_hT=True)
    got = dict(L.scan_bwd(*a, dy.cuda(), softplus=False, **m, want_dh0=True), y=y, hT=hT)
    return {k: (np64(got[k]), v) for k, v in ref.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("case", ["late input", "early gradient", "small state", "small gradient"])
def test_states_that_grow_over_segments(case):
    """Rates of 1 and steps of 1.5: over a segment of 64 tokens a state grows by 2^138, more than a
    float holds, and what enters it is nothing (left padding) or small: the results are finite.

    Steps are multiples of 1/2, so their sums are exact.  A segment's factor is off by the rounding
    of the rate (2^-24) and of the exponent (2^-17 of 138), 2.9e-6 x 2 + 5.3e-6; a token's by 2^-22
    and the sums behind it by some 8 2^-24, over 20 tokens 1.5e-5: 3e-5 holds all."""
    if case == "late input":  # 3 empty segments, then 12 tokens
        r = _growing(204, torch.tensor(1.5).expand(204), list(range(192, 204)), [203])
        names = ("y", "hT", "dC")  # (the gradients before the input are beyond a float)
    elif case == "early gradient":  # the gradient of 12 tokens, nothing behind them
        r = _growing(256, torch.tensor(1.5).expand(256), [255], list(range(12)))
        names = ("y", "hT", "du", "dB", "dh0", "dA", "dC")
    elif case == "small state":  # 2^-100 before 70 tokens of 2^2.16
        r = _growing(70, torch.tensor(1.5).expand(70), [69], [69], h0=2.0 ** -100)
        names = ("y", "hT", "dC")
    else:  # 2^-100 behind a segment of 2^138
        dt = torch.full((128,), 1.5)
        dt[:64] = 0.0
        r = _growing(128, dt, [0], [0], dhT=2.0 ** -100)
        names = ("y", "du", "dh0", "dB")
    for n in names:
        got, ref = r[n]
        assert np.isfinite(ref).all() and np.abs(ref).max() < 3e38, (case, n, "not a test")
        assert np.isfinite(got).all(), (case, n)
        assert np.linalg.norm(got - ref) <= 3e-5 * np.linalg.norm(ref) + 1e-30, (case, n)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,T,n", [(torch.bfloat16, 64, 21, 9), (torch.bfloat16, 13, 40, 33),
                                         (torch.float32, 36, 300, 256), (torch.float32, 5, 9, 1)])
def test_convolution_behind_an_overflow(dtype, D, T, n):
    """The last token of a padded sequence is infinite: its own gradients are not finite, those of
    the tokens behind the end are zeros all the same, and those before the taps' reach are what they
    are without it."""
    K = 4
    g = torch.Generator().manual_seed(T)
    x, dy = (torch.randn(2, T, D, generator=g).to(dtype).cuda() for _ in range(2))
    w, b = torch.randn(D, K, generator=g).cuda(), torch.randn(D, generator=g).cuda()
    lens = torch.tensor([T, n]).cuda()
    want = L.conv_bwd(x, w, dy, b, lens=lens)["dx"]
    x[1, n - 1] = float("inf")
    got = L.conv_bwd(x, w, dy, b, lens=lens)["dx"]
    assert not got[1, n:].any()  # (NaN counts as true)
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1, :max(0, n - K)], want[1, :max(0, n - K)])


class _Stream:  # of a device that no machine need have
    cuda_stream = 0

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_stream_of_another_device_is_refused():
    """Work on a stream goes to that stream's device, which need not reach the tensors' memory."""
    with pytest.raises(ValueError, match="cuda:1"):
        L._on(torch.device("cuda", 0), _Stream(1))


def test_sizes_beyond_32_bits_are_refused():
    """The library's sizes are C ints: a larger one must not arrive there cut off."""
    big = 2 ** 32 + 5
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="meta")
    x, x1, w = e(1, big, 1), e(1, big), e(1, 4)
    calls = [lambda: L.conv_fwd(x, w), lambda: L.conv_bwd(x, w, x), lambda: L.conv_fwd(e(1, 1, big), e(big, 4)),
             lambda: L.conv_step(e(1, 3, big), x1, e(big, 4)),
             lambda: L.scan_fwd(x, x, e(1, 4), e(1, big, 4), e(1, big, 4)),
             lambda: L.scan_bwd(x, x, e(1, 4), e(1, big, 4), e(1, big, 4), x),
             lambda: L.scan_step(e(big, 1, 4), e(big, 1), e(big, 1), e(1, 4), e(big, 4), e(big, 4)),
             lambda: L.block_norm_fwd(e(1, 1, 8), w=e(8), groups=2 ** 32 + 1), lambda: L.block_norm_fwd(x, w=e(1)), lambda: L.block_norm_bwd(x, w=e(1), dout=x),
             lambda: L.block_norm_fwd(e(1, 2 ** 16, 1, 2 ** 16), w=e(2 ** 32))]
    for call in calls:
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def _scan_bwd_args():
    d = L.LzScanDims(2, 4096, 64, 1, 16, L.LZ_BF16, 1)
    return d, [0x7F0000000000 + 4096 * i for i in range(23)]  # never dereferenced


def test_scratch_with_the_forwards_states():
    """The backward that is given the states asks for no room for them, and refuses to go without."""
    d, p = _scan_bwd_args()
    whole, saved, states = (L.lz_layer_workspace_bytes(d, w) for w in
                            (L.LZ_WS_SCAN_BWD, L.LZ_WS_SCAN_BWD_SAVED, L.LZ_WS_SCAN_STATES))
    assert states == 2 * 256 * 64 * 16 * 4 and saved == whole - states > 0
    f = L.load().lz_scan_bwd_saved
    with pytest.raises(L.LzError, match="too small"):
        L._check(f(d, *p, saved - 1, 0))
    with pytest.raises(L.LzError, match="states"):
        L._check(f(d, *p[:12], None, *p[13:], saved, 0))


@pytest.mark.gpu
def test_backward_with_states_takes_no_room_for_them():
    B, T, D, N = 1, 4096, 512, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    u, dt, dy = (torch.randn(B, T, D, generator=g, device="cuda") for _ in range(3))
    bc, A = torch.randn(B, T, N, generator=g, device="cuda"), -torch.ones(D, N, device="cuda")
    st = L.scan_fwd(u, dt, A, bc, bc, want_states=True)[2]

    def peak(states):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        at = torch.cuda.memory_allocated()
        out = L.scan_bwd(u, dt, A, bc, bc, dy, states=states)
        return torch.cuda.max_memory_allocated() - at, out

    (own, a), (given, b) = peak(None), peak(st)
    assert given <= own - 4 * st.numel() + (1 << 20)
    assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,D,N,G", [(torch.bfloat16, 3, 64, 16, 1), (torch.float32, 2, 20, 8, 2),
                                           (torch.bfloat16, 5, 13, 4, 1)])
def test_captured_generation_steps(dtype, B, D, N, G):
    """One token through norm, convolution, scan step and gated norm, captured into a CUDA graph and
    replayed token by token on states that move in place: the bits of the eager calls."""
    g = torch.Generator().manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=g).cuda()
    T, K = 6, 4
    w, b, wc, A, w2 = r(D), r(D), r(D, K), -torch.rand(D, N, generator=g).cuda(), r(D)
    xs, zs, bcs = r(T, B, 1, D).to(dtype), r(T, B, D).to(dtype), r(T, B, 2, G, N).to(dtype)
    hist0, state0 = r(B, K - 1, D).to(dtype), r(B, D, N)
    x, z, bc, hist, state = (torch.empty_like(v) for v in (xs[0], zs[0], bcs[0], hist0, state0))

    def token():
        n, _ = L.block_norm_fwd(x, w=w)
        c = L.conv_step(hist, n[:, 0], wc, b)
        y = L.scan_step(state, c, n[:, 0], A, bc[:, 0], bc[:, 1], Dskip=b, z=z, dt_bias=b)
        return L.block_norm_fwd(y[:, None], w=w, z=z[:, None], r=x, w2=w2)

    def run(step):
        hist.copy_(hist0)
        state.copy_(state0)
        out = []
        for t in range(T):
            for dst, src in ((x, xs[t]), (z, zs[t]), (bc, bcs[t])):
                dst.copy_(src)
            out += [v.clone() for v in step()] + [hist.clone(), state.clone()]
        return out

    want = run(token)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = token()

    def replay():
        graph.replay()
        return got

    assert all(torch.equal(p, q) for p, q in zip(run(replay), want))


@pytest.mark.gpu
def test_slices_off_a_16_byte_boundary_are_refused():
    """One sequence of an odd-sized batch is contiguous and still not where vectors can be stored or
    loaded: the library refuses it; as a strided input it is read."""
    T, D, N = 3, 5, 4
    x, w, o = torch.zeros(2, T, D, device="cuda"), torch.zeros(D, 2, device="cuda"), torch.ones(D, device="cuda")
    bc, A = torch.zeros(1, T, N, device="cuda"), -torch.ones(D, N, device="cuda")
    for call in (lambda v: L.conv_bwd(x[:1], w, v), lambda v: L.scan_bwd(x[:1], x[:1], A, bc, bc, v),
                 lambda v: L.block_norm_bwd(x[:1], w=o, dout=v)):
        with pytest.raises(L.LzError, match="16-byte aligned"):
            call(x[1:])
        call(x[1:].clone())
    L.conv_fwd(x[1:], w)
    L.scan_fwd(x[1:], x[1:], A, bc, bc)
    L.block_norm_fwd(x[1:], w=o)
