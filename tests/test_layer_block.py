"""A layer built of the operators together, as a model would run it: norm ->
projection -> short convolution -> projection of the scan's steps and B, C ->
selective scan -> projection -> gated norm, residual and the next block's norm.
Forward, every gradient, and prompt then single tokens; the projections are
torch products in 32 bits, the reference is autograd in 64 bits."""
import math

import pytest
import torch

import gated_linear_sliding_chunked_b200 as L

pytestmark = pytest.mark.gpu

B, T, DM, D, N, K = 2, 45, 64, 96, 16, 4


def params(seed, heads=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    p = dict(wn=1 + 0.1 * r(DM), Win=r(2 * D, DM) / math.sqrt(DM), wc=r(D, K) / math.sqrt(K),
             bc=0.1 * r(D), Wx=r(D + 2 * N, D) / math.sqrt(D), A=-torch.exp(0.3 * r(D, N)),
             dtb=r(D) - 2, Ds=r(D), Wout=r(DM, D) / math.sqrt(D), wo=1 + 0.1 * r(DM),
             Wg=r(DM, DM) / math.sqrt(DM), s=0.5 + 0.1 * r(DM), w2=1 + 0.1 * r(DM))
    return p, r(B, T, DM)


def plain(p, x, eps=1e-5):
    """The same layer by torch in the given precision."""
    rms = lambda v: v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    silu = torch.nn.functional.silu
    xn = rms(x) * p["wn"]
    xs, z = (xn @ p["Win"].t()).chunk(2, -1)
    pad = torch.cat([xs.new_zeros(xs.shape[0], K - 1, D), xs], 1)
    c = silu(sum(pad[:, j:j + xs.shape[1]] * p["wc"][:, j] for j in range(K)) + p["bc"])
    dt, Bm, Cm = (c @ p["Wx"].t()).split([D, N, N], -1)
    dl = torch.nn.functional.softplus(dt + p["dtb"])
    h, ys = x.new_zeros(x.shape[0], D, N), []
    for t in range(x.shape[1]):
        h = torch.exp(dl[:, t, :, None] * p["A"]) * h + (dl * c)[:, t, :, None] * Bm[:, t, None]
        ys.append((h * Cm[:, t, None]).sum(-1) + p["Ds"] * c[:, t])
    y = torch.stack(ys, 1) * silu(z)
    o = y @ p["Wout"].t()
    out = x + p["s"] * silu(xn @ p["Wg"].t()) * (rms(o) * p["wo"])
    return out, rms(out) * p["w2"]


def forward(p, x):
    """The layer by the library; returns what its backward needs too."""
    xn, _ = L.block_norm_fwd(x, w=p["wn"])
    xz = xn @ p["Win"].t()
    xs, z = xz[..., :D], xz[..., D:]
    c, hist = L.conv_fwd(xs, p["wc"], p["bc"], want_xT=True)
    dbc = c @ p["Wx"].t()
    dt, Bm, Cm = dbc[..., :D], dbc[..., D:D + N], dbc[..., D + N:]
    y, hT, st = L.scan_fwd(c, dt, p["A"], Bm, Cm, Dskip=p["Ds"], z=z, dt_bias=p["dtb"],
                           want_hT=True, want_states=True)
    o = y @ p["Wout"].t()
    gz = xn @ p["Wg"].t()
    out, n = L.block_norm_fwd(o, w=p["wo"], z=gz, s=p["s"], r=x, w2=p["w2"])
    return dict(xn=xn, xs=xs, z=z, c=c, dt=dt, Bm=Bm, Cm=Cm, y=y, st=st, o=o, gz=gz, out=out, n=n,
                hist=hist, hT=hT)


def backward(p, x, f, dout, dn):
    flat = lambda a: a.reshape(-1, a.shape[-1])
    g = {}
    d = L.block_norm_bwd(f["o"], w=p["wo"], z=f["gz"], s=p["s"], w2=p["w2"], out=f["out"],
                         dout=dout, dn=dn, want_dr=True)
    g.update(wo=d["dw"], s=d["ds"], w2=d["dw2"], Wout=flat(d["do"]).t() @ flat(f["y"]),
             Wg=flat(d["dz"]).t() @ flat(f["xn"]))
    sc = L.scan_bwd(f["c"], f["dt"], p["A"], f["Bm"], f["Cm"], d["do"] @ p["Wout"], Dskip=p["Ds"],
                    z=f["z"], dt_bias=p["dtb"], states=f["st"])
    g.update(A=sc["dA"], Ds=sc["dDskip"], dtb=sc["ddt_bias"])
    dbc = torch.cat([sc["ddt"], sc["dB"], sc["dC"]], -1)
    g["Wx"] = flat(dbc).t() @ flat(f["c"])
    cv = L.conv_bwd(f["xs"], p["wc"], sc["du"] + dbc @ p["Wx"], p["bc"])
    g.update(wc=cv["dw"], bc=cv["dbias"])
    dxz = torch.cat([cv["dx"], sc["dz"]], -1)
    g["Win"] = flat(dxz).t() @ flat(f["xn"])
    pre = L.block_norm_bwd(x, w=p["wn"], dout=dxz @ p["Win"] + d["dz"] @ p["Wg"])
    g["wn"] = pre["dw"]
    return pre["do"] + d["dr"], g


def close(name, got, ref, tol):
    err = float((got.double().cpu() - ref).norm() / ref.norm())
    assert err <= tol, (name, err)


def test_layer_forward_and_gradients():
    """In 32 bits each operator is off by some 1e-6 relative (tens of roundings
    of 2^-24, the products' 64 to 128 terms among them); ten of them in a row,
    forward and back, with slopes of order 1: 1e-4 holds all."""
    torch.backends.cuda.matmul.allow_tf32 = False
    p, x = params(0)
    gen = torch.Generator().manual_seed(1)
    dout, dn = (torch.randn(B, T, DM, generator=gen) for _ in range(2))
    ref = {k: v.double().requires_grad_() for k, v in p.items()}
    x64 = x.double().requires_grad_()
    out, n = plain(ref, x64)
    ((out * dout).sum() + (n * dn).sum()).backward()
    dev = {k: v.cuda() for k, v in p.items()}
    xd = x.cuda()
    f = forward(dev, xd)
    close("out", f["out"], out.detach(), 1e-4)
    close("n", f["n"], n.detach(), 1e-4)
    dx, g = backward(dev, xd, f, dout.cuda(), dn.cuda())
    close("x", dx, x64.grad, 1e-4)
    for k in p:
        close(k, g[k], ref[k].grad, 1e-4)


def test_layer_prompt_then_single_tokens():
    """The prompt's histories and states continue with the single-token calls:
    every output equals the whole sequence's."""
    torch.backends.cuda.matmul.allow_tf32 = False
    p, x = params(2)
    out, n = plain({k: v.double() for k, v in p.items()}, x.double())
    dev, xd, T0 = {k: v.cuda() for k, v in p.items()}, x.cuda(), 30
    f = forward(dev, xd[:, :T0].contiguous())
    hist, h = f["hist"], f["hT"]
    outs = [f["out"]]
    for t in range(T0, T):
        xt = xd[:, t:t + 1].contiguous()
        xn, _ = L.block_norm_fwd(xt, w=dev["wn"])
        xz = xn[:, 0] @ dev["Win"].t()
        c = L.conv_step(hist, xz[:, :D], dev["wc"], dev["bc"])
        dbc = c @ dev["Wx"].t()
        y = L.scan_step(h, c, dbc[:, :D], dev["A"], dbc[:, D:D + N], dbc[:, D + N:],
                        Dskip=dev["Ds"], z=xz[:, D:], dt_bias=dev["dtb"])
        o = (y @ dev["Wout"].t())[:, None]
        outs.append(L.block_norm_fwd(o, w=dev["wo"], z=xn @ dev["Wg"].t(), s=dev["s"], r=xt,
                                     w2=dev["w2"])[0])
    close("out", torch.cat(outs, 1), out, 1e-4)


def test_attention_output_through_the_gated_norm():
    """The hybrid attention's output by heads, normed a head and gated into
    rows for the output projection, with the gradient back to it."""
    H, d, w = 4, 128, 16
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g)
    q, k, v = ((r(B, H, T, d) / math.sqrt(d)).bfloat16().cuda() for _ in range(3))
    gate = (torch.nn.functional.logsigmoid(r(B, H, T, d)) / 16).cuda()
    mk, mv = r(H, 2, d).bfloat16().cuda(), r(H, 2, d).bfloat16().cuda()
    wn, z = (1 + 0.1 * r(H * d)).cuda(), r(B, T, H * d).bfloat16().cuda()
    o = L.hybrid_fwd(q, k, v, gate, mk, mv, w=w, alpha=0.5)["o"]
    out, _ = L.block_norm_fwd(o, w=wn, z=z, groups=H)
    dout = r(B, T, H * d).bfloat16().cuda()
    got = L.block_norm_bwd(o, w=wn, z=z, dout=dout, groups=H)
    o64 = o.double().requires_grad_()
    n = o64 * torch.rsqrt((o64 * o64).mean(-1, keepdim=True) + 1e-5)
    ref = n.transpose(1, 2).reshape(B, T, -1) * wn.double() * torch.nn.functional.silu(z.double())
    ref.backward(dout.double())
    # one rounding to bf16 (2^-8 of each value) over everything else
    close("out", out, ref.detach().cpu(), 2.0 ** -8)
    close("do", got["do"], o64.grad.cpu(), 2.0 ** -8)


def test_calls_on_another_stream_keep_their_scratch():
    """Calls on a side stream while the current one allocates and fills memory
    of the same sizes: what the side stream's kernels still use is not handed
    out (their scratch is freed as soon as the call returns)."""
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g).cuda()
    x, w, dy = r(2, 3000, 256), r(256, 4), r(2, 3000, 256)
    o, wn = r(1, 4000, 512), r(512)
    dt, A, bc = r(2, 3000, 256), -torch.rand(256, 16, generator=g).cuda(), r(2, 3000, 16)

    def calls(stream=None):
        out = [L.conv_bwd(x, w, dy, stream=stream), L.block_norm_bwd(o, w=wn, dout=o, stream=stream),
               L.scan_bwd(x, dt, A, bc, bc, dy, stream=stream)]
        return [t for d in out for t in d.values() if t is not None]

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)  # the side stream's work starts late
        side.wait_stream(torch.cuda.current_stream())
        got = calls(handle)
        for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24):
            for _ in range(4):
                torch.full((n,), float("nan"), device="cuda")
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("D", [48, 1024, 2056, 37])
def test_captured_norms_and_convolutions_replay(D):
    """Forward and backward in one CUDA graph, replayed on new inputs: the bits of the eager calls."""
    gen = torch.Generator().manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    make = lambda: dict(x=r(2, 21, D).bfloat16(), z=r(2, 21, D).bfloat16(), w=r(D), wc=r(D, 4), b=r(D),
                        x0=r(2, 3, D).bfloat16(), dy=r(2, 21, D).bfloat16())

    def call(v):
        y, xT = L.conv_fwd(v["x"], v["wc"], v["b"], v["x0"], want_xT=True)
        out, n = L.block_norm_fwd(y, w=v["w"], z=v["z"], r=v["x"], w2=v["b"])
        g = L.block_norm_bwd(y, w=v["w"], z=v["z"], w2=v["b"], out=out, dn=v["dy"], want_dr=True)
        c = L.conv_bwd(v["x"], v["wc"], g["do"], v["b"], v["x0"], want_dx0=True)
        return [y, xT, out, n] + [t for d in (g, c) for t in d.values() if t is not None]

    a, b = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(a)
    want = call(b)
    for k in a:
        a[k].copy_(b[k])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_rows_beyond_32_bit_offsets():
    """The second sequence stands more than 2^32 elements behind the first: the results are those of
    contiguous inputs, bit for bit."""
    T, D, N = 70, 48, 8
    gen = torch.Generator().manual_seed(5)
    gap = (1 << 32) + 64
    buf = torch.empty(gap + 8 * T * D, dtype=torch.bfloat16, device="cuda")
    far = []

    def place(*shape):
        x = torch.randn(2, T, *shape, generator=gen).bfloat16().cuda()
        width = x[0, 0].numel()
        v = buf[len(far) * T * D:].as_strided((2, T) + shape, (gap, width) + x.stride()[2:])
        v.copy_(x)
        far.append(v)
        return x, v

    (x, xv), (dt, dtv), (z, zv), (Bm, Bv), (Cm, Cv) = place(D), place(D), place(D), place(N), place(N)
    f = lambda *s: torch.randn(*s, generator=gen).cuda()
    w, b, A = f(D, 4), f(D), -torch.rand(D, N, generator=gen).cuda()
    dy = f(2, T, D).bfloat16()

    def call(x, dt, z, Bm, Cm):
        y, _ = L.conv_fwd(x, w, b)
        c = L.conv_bwd(x, w, dy, b)
        out, n = L.block_norm_fwd(x, w=b, z=z, r=dt, w2=b)
        g = L.block_norm_bwd(x, w=b, z=z, w2=b, out=out, dn=dy, want_dr=True)
        s, hT = L.scan_fwd(x, dt, A, Bm, Cm, z=z, want_hT=True)
        sg = L.scan_bwd(x, dt, A, Bm, Cm, dy, z=z)
        return [y, out, n, s, hT] + [t for d in (c, g, sg) for t in d.values() if t is not None]

    assert all(torch.equal(p, q) for p, q in zip(call(x, dt, z, Bm, Cm), call(xv, dtv, zv, Bv, Cv)))
