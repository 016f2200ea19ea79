"""The operators around the scan as they are used: together in a block's training step and decode
loop, captured into HIP graphs, on other streams, and from several host threads."""
import threading

import numpy as np
import pytest

import block_ref as ref
from gpu_helpers import say
from test_gpu_graph import capture, eager_noise, nan_fill
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def tensors(dev, seed, *shapes, dt=None):
    import torch
    gen = torch.Generator(device="cpu").manual_seed(seed)
    return [torch.randn(*s, generator=gen).to(dev, dt or torch.float32) for s in shapes]


def gates(t):
    import torch
    return torch.nn.functional.logsigmoid(t + 3.0)


def np64(t):
    return t.double().cpu().numpy()


def test_training_step_of_a_block(dev):
    """A residual block with a recurrence, fp32: r = x + res, y = norm(r), z = recurrence(y), and back:
    the gradients of <dZ, z> + <dR, r> for x, weight, gates and state, then their norm and clipping,
    against the fp64 forms chained the same way."""
    import torch
    B, H, T, d = 2, 3, 400, 64
    x, res, dz, dr, gl = tensors(dev, 1, *[(B, H, T, d)] * 5)
    w, = tensors(dev, 2, (d,))
    h0, = tensors(dev, 3, (B, H, d))
    g = gates(gl)
    y, r = ttt.rmsnorm_fwd(x, w, res, EPS)
    z, hT = ttt.gated_fwd(y, g, h0)
    dy, dg, dh0 = ttt.gated_bwd(g, z, dz, h0, None)
    dx, dw = ttt.rmsnorm_bwd(r, w, dy, dr, EPS)
    outs, norm = ttt.clip_grad_norm([dx, dw, dg, dh0], 1.0)
    torch.cuda.synchronize()

    flat = lambda t: np64(t).reshape(B * H, T, d)  # noqa: E731
    yy, rr = ref.rmsnorm(flat(x), np64(w), flat(res), EPS)
    h = np64(h0).reshape(B * H, d)
    zz = ref.gated(yy, flat(g), h)
    dyy, dgg, dhh = ref.gated_bwd(flat(g), zz, h, flat(dz), np.zeros_like(h))
    dxx, dww = ref.rmsnorm_bwd(rr.reshape(-1, d), np64(w), dyy.reshape(-1, d), flat(dr).reshape(-1, d), EPS)
    want, n = ref.clip([dxx, dww, dgg, dhh], 1.0, EPS)
    # each stage is good to a few hundred fp32 steps of its largest values; four stages
    say("norm %.6g, %.6g" % (norm.item(), n))
    assert abs(norm.item() - n) <= 2000 * ref.U * n
    for got, v, name in zip(outs, want, ("dx", "dw", "dg", "dh0")):
        err = np.abs(np64(got).reshape(v.shape) - v).max() / np.abs(v).max()
        say(name, "%.3g" % err)
        assert err <= 2000 * ref.U, name


def test_decode_loop_is_the_sequence(dev):
    """Norm and recurrence token by token, next to the fast-weight step: the same as over the whole
    sequence at once (bf16; each stage rounds alike, the states' order of additions differs)."""
    import torch
    B, H, T, d, chunk = 2, 3, 37, 64, 16
    x, gl, res = tensors(dev, 5, *[(B, H, T, d)] * 3, dt=torch.bfloat16)
    w, = tensors(dev, 6, (d,))
    g = gates(gl)
    y, r = ttt.rmsnorm_fwd(x, w, res, EPS)
    z, hT = ttt.gated_fwd(y, g)
    W = torch.zeros(B, H, d, d, device=dev)
    q = torch.nn.functional.normalize(y.float(), dim=-1).to(torch.bfloat16)
    out, WT = ttt.linear_fwd(q, q, z, None, W, chunk, 0.1)
    h, Wc, Gs, pos = torch.zeros(B, H, d, device=dev), W.clone(), torch.zeros_like(W), 0
    zs, os, rs = [], [], []
    for t in range(T):
        at = lambda a: a[:, :, t:t + 1].contiguous()  # noqa: E731
        yt, rt = ttt.rmsnorm_fwd(at(x), w, at(res), EPS)
        assert torch.equal(yt, at(y)) and torch.equal(rt, at(r))
        zt = ttt.gated_step(yt, at(g), h)
        ot, pos = ttt.linear_step(at(q), at(q), at(z), None, Wc, Gs, pos, chunk, 0.1)
        zs.append(zt)
        os.append(ot)
    torch.cuda.synchronize()
    yy, gg = np64(y).reshape(B * H, T, d), np64(g).reshape(B * H, T, d)
    h0 = np.zeros((B * H, d))
    want, bound = ref.gated(yy, gg, h0), ref.gated_bound(yy, gg, h0)
    for got in (z, torch.cat(zs, 2)):
        assert ref.within(np64(got).reshape(B * H, T, d), want, bound, "bf16")[0]
    for got in (hT, h):
        assert ref.within(np64(got).reshape(B * H, d), want[:, -1], bound[:, -1], "f32")[0]
    err = (torch.cat(os, 2).float() - out.float()).abs().max() / out.float().abs().max()
    assert err < 2e-2          # the scan's own tolerance for bf16


def test_quantized_norm_feeds_a_projection(dev):
    """Y8 * scale is what a projection reads: within one rounding of the unquantized output."""
    import torch
    x, res = tensors(dev, 7, (64, 768), (64, 768), dt=torch.bfloat16)
    w, = tensors(dev, 8, (768,))
    y, r = ttt.rmsnorm_fwd(x, w, res, EPS)
    y8, scale, r8 = ttt.rmsnorm_q8_fwd(x, w, res, EPS)
    assert torch.equal(r, r8)
    back = y8.float() * scale[:, None]
    room = torch.maximum(y.float().abs() * (2.0 ** -4 + 2.0 ** -8) * 1.01, scale[:, None] * 2.0 ** -10)
    assert ((back - y.float()).abs() <= room).all()


def calls(dev, long):
    """(name, outputs, fn) of one call of each operator, with its outputs and workspace set up."""
    import torch
    B, H, T, d = (2, 3, 3000, 64) if long else (2, 3, 70, 83)
    bf = torch.bfloat16
    X, gl, dZ = tensors(dev, 11, *[(B, H, T, d)] * 3, dt=bf)
    G = gates(gl)
    h0, dh = tensors(dev, 12, (B, H, d), (B, H, d))
    Z, hT, dX, dG, dh0 = (torch.empty_like(t) for t in (X, h0, X, X, h0))
    n = max(1, ttt.gated_workspace_bytes(B, H, T, d, 1))
    ws = [torch.empty(n, dtype=torch.uint8, device=dev) for _ in range(2)]
    Zin = ttt.gated_fwd(X, G, h0)[0]
    rows, D = (3000, 768) if long else (9, 100)
    x, res, dY = tensors(dev, 13, *[(rows, D)] * 3, dt=bf)
    w, = tensors(dev, 14, (D,))
    Y, R, dx = (torch.empty_like(x) for _ in range(3))
    Y8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=dev)
    sc, dw = torch.empty(rows, device=dev), torch.empty(D, device=dev)
    wr = torch.empty(ttt.rmsnorm_bwd_workspace_bytes(rows, D, 1), dtype=torch.uint8, device=dev)
    grads = tensors(dev, 15, *[((40000 if long else 50) + k,) for k in range(5)])
    outs = [torch.empty_like(g) for g in grads]
    norm = torch.empty(1, device=dev)
    wc = torch.empty(ttt.clip_workspace_bytes(), dtype=torch.uint8, device=dev)
    return [
        ("gated_fwd", [Z, hT], lambda: ttt.gated_fwd(X, G, h0, Z=Z, h_out=hT, workspace=ws[0])),
        ("gated_bwd", [dX, dG, dh0], lambda: ttt.gated_bwd(G, Zin, dZ, h0, dh, dX=dX, dG=dG, dh0=dh0,
                                                           workspace=ws[1])),
        ("rmsnorm_fwd", [Y], lambda: ttt.rmsnorm_fwd(x, w, None, EPS, Y=Y)),
        ("rmsnorm_q8_fwd", [Y8.view(torch.uint8), sc, R],
         lambda: ttt.rmsnorm_q8_fwd(x, w, res, EPS, Y8=Y8, scale=sc, R=R)),
        ("rmsnorm_bwd", [dx, dw], lambda: ttt.rmsnorm_bwd(x, w, dY, res, EPS, dX=dx, dweight=dw,
                                                          workspace=wr)),
        ("clip_grad_norm", outs + [norm], lambda: ttt.clip_grad_norm(grads, 1.0, outs=outs, norm=norm,
                                                                     workspace=wc)),
    ]


def wipe(outs):
    import torch
    for t in outs:
        if t.dtype == torch.uint8:
            t.fill_(85)
        else:
            nan_fill(t)


@pytest.mark.parametrize("long", [False, True])
def test_graphs_replay(dev, long):
    import torch
    for name, outs, fn in calls(dev, long):
        say("case", name)
        fn()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        g = capture(fn)
        for k in range(4):
            wipe(outs)
            eager_noise(dev)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), (name, k)


def test_one_graph_of_all(dev):
    """A step of every operator in one graph, replayed on new inputs' values as well."""
    import torch
    every = calls(dev, True)
    for _, _, fn in every:
        fn()
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, outs, _ in every]

    def step():
        for _, _, fn in every:
            fn()

    g = capture(step)
    for k in range(3):
        for _, outs, _ in every:
            wipe(outs)
        eager_noise(dev)
        g.replay()
        torch.cuda.synchronize()
        for (name, outs, _), w in zip(every, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, w)), (name, k)


def test_other_streams(dev):
    """Calls with `stream` given, on tensors made ready for it, several streams at once; the binding's
    own workspaces are not handed to another stream while a call runs."""
    import torch
    X, gl, dZ = tensors(dev, 21, *[(1, 16, 6000, 64)] * 3)
    G = gates(gl)
    Z, hT = ttt.gated_fwd(X, G)
    back = ttt.gated_bwd(G, Z, dZ)
    grads = tensors(dev, 22, (300000,), (70001,))
    outs, norm = ttt.clip_grad_norm(grads, 1.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(4):
        got = []
        for s in streams:
            got.append((s, ttt.gated_fwd(X, G, stream=s), ttt.gated_bwd(G, Z, dZ, stream=s),
                        ttt.clip_grad_norm(grads, 1.0, stream=s)))
        for _ in range(5):          # work on the current stream that would take a freed workspace
            torch.empty(1 << 20, device=dev).fill_(float("nan"))
        torch.cuda.synchronize()
        for s, (z, h), b, (o, n) in got:
            assert torch.equal(z, Z) and torch.equal(h, hT)
            assert all(torch.equal(p, q) for p, q in zip(b, back))
            assert torch.equal(n, norm) and all(torch.equal(p, q) for p, q in zip(o, outs))


def test_host_threads(dev):
    import torch
    X, gl = tensors(dev, 31, *[(1, 8, 5000, 64)] * 2)
    G = gates(gl)
    Z, hT = ttt.gated_fwd(X, G)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(10):
            z, h = ttt.gated_fwd(X, G, stream=s)
            s.synchronize()
            if not (torch.equal(z, Z) and torch.equal(h, hT)):
                bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_binding_refuses(dev):
    import torch
    X, G = tensors(dev, 41, *[(1, 2, 8, 16)] * 2)
    h = torch.zeros(1, 2, 16, device=dev)
    for bad in (G.bfloat16(), G[:, :, :4], G.transpose(2, 3), G.cpu()):
        with pytest.raises(ValueError):
            ttt.gated_fwd(X, bad)
        with pytest.raises(ValueError):
            ttt.gated_bwd(G, X, bad)
    with pytest.raises(ValueError):
        ttt.gated_fwd(X, G, h.bfloat16())
    with pytest.raises(ValueError):
        ttt.gated_step(X, G, h[:, :1])
    with pytest.raises(TypeError):
        ttt.gated_fwd(X.half(), G.half())
    with pytest.raises(ttt.TTTError):
        ttt.gated_fwd(X, G, Z=X)
    # contiguous, but not where a 16-byte access may start
    off = torch.zeros(X.numel() + 1, device=dev)[1:].view(X.shape)
    for call in (lambda: ttt.gated_fwd(off, G), lambda: ttt.gated_fwd(X, off),
                 lambda: ttt.gated_step(X, off, h), lambda: ttt.gated_bwd(G, X, off),
                 lambda: ttt.rmsnorm_fwd(off), lambda: ttt.rmsnorm_q8_fwd(X, None, off),
                 lambda: ttt.rmsnorm_bwd(X, None, off)):
        with pytest.raises(ttt.TTTError):
            call()
    big = ttt.gated_workspace_bytes(1, 2, 4096, 16, 0)
    XL, GL = (t.repeat(1, 1, 512, 1) for t in (X, G))
    for ws in (torch.empty(big, dtype=torch.uint8), torch.empty(big, device=dev),
               torch.empty(2 * big, dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError):
            ttt.gated_fwd(XL, GL, workspace=ws)
    with pytest.raises(ttt.TTTError):
        ttt.gated_fwd(XL, GL, workspace=torch.empty(big - 1, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        ttt.rmsnorm_fwd(X, torch.ones(8, device=dev))
    with pytest.raises(ValueError):
        ttt.rmsnorm_fwd(X, None, X.bfloat16())
    with pytest.raises(ttt.TTTError):
        ttt.rmsnorm_fwd(X, None, None, 0.0)
    with pytest.raises(ValueError):
        ttt.clip_grad_norm([X], 1.0, outs=[X, X])
    with pytest.raises(ttt.TTTError):
        ttt.clip_grad_norm([X, X], 1.0, outs=[X, X])
    with pytest.raises(ValueError):
        ttt.clip_grad_norm([X.transpose(2, 3)], 1.0)
    with pytest.raises(ttt.TTTError):
        ttt.clip_grad_norm([X], -1.0)
    torch.cuda.synchronize()
