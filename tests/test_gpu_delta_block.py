"""The gated delta rule with the group norm and dropout behind it as they are used: together in a
layer's training step and decode loop, captured into HIP graphs, on other streams, from several host
threads, and with tensors past 2^31 elements."""
import threading

import numpy as np
import pytest

import block_ref
import delta_ref as ref
from gpu_helpers import say
from test_gpu_graph import capture, eager_noise, nan_fill
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu

EPS = 1e-5


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


def np64(t):
    return t.double().cpu().numpy()


def unit(t):
    """Rows of unit length by the RMS norm: x / |x| = rmsnorm(x) / sqrt(d)."""
    import torch
    d = t.shape[-1]
    w = torch.full((d,), d ** -0.5, device=t.device)
    return ttt.rmsnorm_fwd(t, w, eps=1e-6)[0], w


def test_training_step_of_a_layer(dev):
    """Tokens first: keys and queries to unit length, the delta rule, the norm of every head's output
    with SiLU, dropout and the residual; and the whole way back. fp32, against the fp64 forms chained
    the same way."""
    import torch
    B, T, H, d, p = 2, 150, 3, 64, 0.25
    k, q, v, res, dy = tensors(dev, 1, *[(B, T, H, d)] * 5)
    el, gl = tensors(dev, 2, (B, T, H), (B, T, H))
    w, b = tensors(dev, 3, (H * d,), (H * d,))
    W0, = tensors(dev, 4, (B, H, d, d))
    w, eta, g = 1 + 0.2 * w, torch.sigmoid(el), torch.nn.functional.logsigmoid(gl + 3)
    rng = torch.tensor([77, 1000], device=dev)
    lay = ttt.LAYOUT_BTHD
    K, wu = unit(k)
    Q, _ = unit(q)
    z, WT = ttt.delta_fwd(K, Q, v, eta, g, W0, layout=lay)
    zf = z.view(B * T, H * d)
    n, mean, rstd = ttt.groupnorm_fwd(zf, H, w, b, EPS, ttt.ACT_SILU)
    y = ttt.dropout(n, p, rng, res.view(B * T, H * d))
    dn = ttt.dropout(dy.view(B * T, H * d), p, rng)
    dz, dw, db = ttt.groupnorm_bwd(zf, H, w, b, dn, mean, rstd, ttt.ACT_SILU)
    dK, dQ, dv, deta, dg, dW0 = ttt.delta_bwd(K, Q, v, eta, g, W0, dz.view(B, T, H, d), layout=lay)
    dk = ttt.rmsnorm_bwd(k, wu, dK)[0]
    torch.cuda.synchronize()

    heads = lambda t: np.swapaxes(np64(t), 1, 2).reshape((B * H, T) + tuple(t.shape[3:]))  # noqa: E731
    flat = lambda a: np.swapaxes(a.reshape(B, H, T, d), 1, 2).reshape(B * T, 1, H * d)  # noqa: E731
    back = lambda a: np.swapaxes(a.reshape(B, T, H, d), 1, 2).reshape(B * H, T, d)  # noqa: E731
    wun = np64(wu)
    KK, QQ = (block_ref.rmsnorm(heads(t), wun, None, 1e-6)[0] for t in (k, q))
    W00 = np64(W0).reshape(B * H, d, d)
    args = (KK, QQ, heads(v), heads(eta), heads(g), W00)
    zz = ref.delta(*args)[0]
    nn, mm, rr = ref.groupnorm(flat(zz), H, np64(w), np64(b), EPS, "silu")[:3]
    keep = ref.keep_mask(B * T * H * d, p, 77, 1000).reshape(nn.shape)
    yy = np.where(keep, nn / (1 - p), 0) + np64(res).reshape(nn.shape)
    dnn = np.where(keep, np64(dy).reshape(nn.shape) / (1 - p), 0)
    dzz, dww, dbb = ref.groupnorm_bwd(flat(zz), H, np64(w), np64(b), dnn, mm, rr, "silu")[0]
    want = ref.delta_bwd(*args, back(dzz), np.zeros_like(W00))
    dkk = block_ref.rmsnorm_bwd(heads(k).reshape(-1, d), wun, want[0].reshape(-1, d), None, 1e-6)[0]
    got = [(y, yy), (dw, dww), (db, dbb), (heads(dQ), want[1]), (heads(dv), want[2]), (heads(deta), want[3]),
           (heads(dg), want[4]), (dW0, want[5]), (heads(dk), dkk.reshape(B * H, T, d))]
    # each stage is good to some hundred fp32 steps of its largest values (430 for the delta rule),
    # and the next carries that on; five stages
    for i, (a, c) in enumerate(got):
        a = np64(a) if not isinstance(a, np.ndarray) else a
        err = np.abs(a.reshape(c.shape) - c).max() / np.abs(c).max()
        say(i, "%.3g" % err)
        assert err <= 4000 * ref.U, i


def test_decode_loop_is_the_sequence(dev):
    """The delta rule and the norm token by token from a prefill's state: as over the whole sequence."""
    import torch
    B, T, H, Hk, d, dv, pre = 2, 100, 4, 2, 64, 83, 70
    k, q = tensors(dev, 5, *[(B, T, Hk, d)] * 2)
    v, = tensors(dev, 6, (B, T, H, dv))
    el, gl = tensors(dev, 7, (B, T, H), (B, T, H))
    K, Q, eta, g = unit(k)[0], unit(q)[0], torch.sigmoid(el), torch.nn.functional.logsigmoid(gl + 3)
    lay = ttt.LAYOUT_BTHD
    whole, WT = ttt.delta_fwd(K, Q, v, eta, g, layout=lay)
    n_whole = ttt.groupnorm_fwd(whole.reshape(B * T, H * dv), H, act=ttt.ACT_SILU)[0].view(B, T, H * dv)
    cut = lambda t, s: t[:, s].clone()  # noqa: E731
    head = slice(0, pre)
    z, W = ttt.delta_fwd(*[cut(t, head) for t in (K, Q, v, eta, g)], layout=lay)
    zs, ns = [z], []
    for t in range(pre, T):
        zt = ttt.delta_step(*[cut(x, slice(t, t + 1)) for x in (K, Q, v, eta, g)], W, layout=lay)
        zs.append(zt)
        ns.append(ttt.groupnorm_fwd(zt.view(B, H * dv), H, act=ttt.ACT_SILU)[0])
    rel = 2 * ref.delta_rel(T, d, dv)
    assert (torch.cat(zs, 1) - whole).abs().max() <= rel * whole.abs().max()
    assert (W - WT).abs().max() <= rel * WT.abs().max()
    # (the norm divides by a head's spread, which is about a quarter of the largest value)
    assert (torch.stack(ns, 1) - n_whole[:, pre:]).abs().max() <= 8 * rel * n_whole.abs().max()


def calls(dev, long):
    """(name, outputs, fn) of one call of each operator, with its outputs and workspace set up."""
    import torch
    B, H, T, d = (1, 4, 2500, 64) if long else (2, 3, 70, 50)
    bf = torch.bfloat16
    K, Q, V, dZ = tensors(dev, 11, *[(B, H, T, d)] * 4, dt=bf)
    K, Q = (torch.nn.functional.normalize(t.float(), dim=-1).to(bf) for t in (K, Q))
    el, gl = tensors(dev, 12, (B, H, T), (B, H, T))
    eta, g = torch.sigmoid(el), torch.nn.functional.logsigmoid(gl + 3)
    W0, dW = tensors(dev, 13, *[(B, H, d, d)] * 2)
    Z, W, dK, dQ, dV, de, dg, dW0, Zs, Ws = (torch.empty_like(t) for t in (V, W0, K, Q, V, eta, g, W0, V, W0))
    byte = lambda n: torch.empty(max(1, n), dtype=torch.uint8, device=dev)  # noqa: E731
    wf = byte(ttt.delta_workspace_bytes(B, H, H, T, d, d, 1))
    wb = byte(ttt.delta_bwd_workspace_bytes(B, H, H, T, d, d, 1))
    N, S, C, G = (3, 900, 96, 4) if long else (50, 1, 96, 4)
    X, dY = tensors(dev, 14, *[(N, S, C)] * 2, dt=bf)
    w, b = tensors(dev, 15, (C,), (C,))
    mean0, rstd0 = ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_GELU)[1:]
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    mean, rstd, dw, db = (torch.empty_like(t) for t in (mean0, rstd0, w, b))
    gf, gb = byte(ttt.groupnorm_workspace_bytes(N, S, C, G, 1)), byte(ttt.groupnorm_bwd_workspace_bytes(N, S, C, G, 1))
    rng = torch.tensor([5, 6], device=dev)
    D = torch.empty_like(X)

    def step():
        Ws.copy_(W0)
        ttt.delta_step(K, Q, V, eta, g, Ws, Z=Zs)

    return [
        ("delta_fwd", [Z, W], lambda: ttt.delta_fwd(K, Q, V, eta, g, W0, Z=Z, W_out=W, workspace=wf)),
        ("delta_bwd", [dK, dQ, dV, de, dg, dW0],
         lambda: ttt.delta_bwd(K, Q, V, eta, g, W0, dZ, dW, dK=dK, dQ=dQ, dV=dV, deta=de, dg=dg, dW0=dW0,
                               workspace=wb)),
        ("delta_step", [Zs, Ws], step),
        ("groupnorm_fwd", [Y, mean, rstd],
         lambda: ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_GELU, Y=Y, mean=mean, rstd=rstd, workspace=gf)),
        ("groupnorm_bwd", [dX, dw, db],
         lambda: ttt.groupnorm_bwd(X, G, w, b, dY, mean0, rstd0, ttt.ACT_GELU, dX=dX, dweight=dw, dbias=db,
                                   workspace=gb)),
        ("dropout", [D], lambda: ttt.dropout(X, 0.3, rng, dY, Y=D)),
    ]


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
            nan_fill(*outs)
            eager_noise(dev)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), (name, k)


def test_one_graph_of_all(dev):
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
            nan_fill(*outs)
        eager_noise(dev)
        g.replay()
        torch.cuda.synchronize()
        for (name, outs, _), w in zip(every, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, w)), (name, k)


def test_a_graph_draws_anew(dev):
    """A captured dropout reads its counter at each replay."""
    import torch
    X, = tensors(dev, 16, (5000,))
    rng = torch.tensor([9, 0], device=dev)
    Y = torch.empty_like(X)
    g = capture(lambda: ttt.dropout(X, 0.5, rng, Y=Y))
    for first in (0, 1250, 2500):
        rng[1] = first
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, ttt.dropout(X, 0.5, rng))
        assert np.array_equal((Y != 0).cpu().numpy(), ref.keep_mask(5000, 0.5, 9, first))


def test_other_streams(dev):
    """Calls with `stream` given, several streams at once, with workspaces of the binding's own."""
    import torch
    K, Q, V, dZ = tensors(dev, 21, *[(1, 8, 3000, 64)] * 4)
    K, Q = (torch.nn.functional.normalize(t, dim=-1) for t in (K, Q))
    eta, g = torch.full((1, 8, 3000), 0.5, device=dev), torch.full((1, 8, 3000), -0.1, device=dev)
    X, dY = tensors(dev, 22, *[(4, 2000, 64)] * 2)
    w, = tensors(dev, 23, (64,))
    rng = torch.tensor([1, 2], device=dev)
    every = [lambda s: ttt.delta_fwd(K, Q, V, eta, g, stream=s), lambda s: ttt.delta_bwd(K, Q, V, eta, g, None, dZ, stream=s),
             lambda s: ttt.groupnorm_fwd(X, 4, w, w, stream=s), lambda s: (ttt.dropout(X, 0.5, rng, stream=s),)]
    want = [f(None) for f in every]
    mean, rstd = want[2][1:]
    every.append(lambda s: ttt.groupnorm_bwd(X, 4, w, w, dY, mean, rstd, stream=s))
    want.append(every[-1](None))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        got = [[f(s) for f in every] for s in streams]
        for _ in range(5):          # work on the current stream that would take a freed workspace
            torch.empty(1 << 22, device=dev).fill_(float("nan"))
        torch.cuda.synchronize()
        for outs in got:
            for a, b in zip(outs, want):
                assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_host_threads(dev):
    import torch
    every = calls(dev, False)
    torch.cuda.synchronize()
    K, Q, V, dZ = tensors(dev, 31, *[(1, 4, 500, 64)] * 4)
    K, Q = (torch.nn.functional.normalize(t, dim=-1) for t in (K, Q))
    eta = torch.full((1, 4, 500), 0.5, device=dev)
    want = ttt.delta_fwd(K, Q, V, eta) + ttt.delta_bwd(K, Q, V, eta, None, None, dZ)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(10):
            got = ttt.delta_fwd(K, Q, V, eta, stream=s) + ttt.delta_bwd(K, Q, V, eta, None, None, dZ, stream=s)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and len(every) == 6


def test_binding_refuses(dev):
    import torch
    K, V = tensors(dev, 41, *[(1, 2, 40, 16)] * 2)
    eta = torch.full((1, 2, 40), 0.5, device=dev)
    W = torch.zeros(1, 2, 16, 16, device=dev)
    for bad in (K.bfloat16(), K[:, :, :4], K.transpose(2, 3), K.cpu(), K[:, :1]):
        with pytest.raises(ValueError):
            ttt.delta_fwd(K, bad, V, eta)
        with pytest.raises(ValueError):
            ttt.delta_bwd(K, K, V, eta, None, None, bad)
    for bad in (eta.bfloat16(), eta[:, :, :3], eta.cpu()):
        with pytest.raises(ValueError):
            ttt.delta_fwd(K, K, V, bad)
        with pytest.raises(ValueError):
            ttt.delta_fwd(K, K, V, eta, bad)
    with pytest.raises(ValueError):                 # three heads of values for two of keys
        ttt.delta_fwd(K, K, torch.zeros(1, 3, 40, 16, device=dev), eta)
    with pytest.raises(ValueError):
        ttt.delta_step(K, K, V, eta, None, W[:, :1])
    with pytest.raises(TypeError):
        ttt.delta_fwd(K.half(), K.half(), V.half(), eta)
    wide = torch.zeros(1, 1, 40, 129, device=dev)
    with pytest.raises(ttt.TTTError):
        ttt.delta_fwd(wide, wide, wide, eta[:, :1].contiguous())
    with pytest.raises(ttt.TTTError):
        ttt.delta_fwd(K, K, V, eta, Z=V)
    off = torch.zeros(K.numel() + 1, device=dev)[1:].view(K.shape)
    for call in (lambda: ttt.delta_fwd(off, K, V, eta), lambda: ttt.delta_step(K, off, V, eta, None, W),
                 lambda: ttt.delta_bwd(K, K, off, eta, None, None, V), lambda: ttt.groupnorm_fwd(off, 2),
                 lambda: ttt.dropout(off, 0.1, torch.zeros(2, dtype=torch.int64, device=dev))):
        with pytest.raises(ttt.TTTError):
            call()
    need = ttt.delta_workspace_bytes(1, 2, 2, 40, 16, 16, 0)
    with pytest.raises(ttt.TTTError):
        ttt.delta_fwd(K, K, V, eta, workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        ttt.delta_fwd(K, K, V, eta, workspace=torch.empty(need, device=dev))
    with pytest.raises(ttt.TTTError):
        ttt.groupnorm_fwd(K, 4, eps=0.0)
    with pytest.raises(ttt.TTTError):
        ttt.groupnorm_fwd(K, 4, act=7)
    with pytest.raises(ValueError):
        ttt.groupnorm_bwd(K, 4, None, None, V, eta, eta)
    with pytest.raises(ValueError):
        ttt.dropout(K, 0.1, torch.zeros(2, device=dev))
    with pytest.raises(ttt.TTTError):
        ttt.dropout(K, 1.0, torch.zeros(2, dtype=torch.int64, device=dev))


def test_groupnorm_and_dropout_past_32_bits(dev):
    """More than 2^32 elements: the last rows are as they are alone."""
    import torch
    rows, C = (1 << 21) + 5, 2048
    X = torch.empty(rows, C, dtype=torch.bfloat16, device=dev)
    X[:-4].fill_(1.0)
    X[-4:], = tensors(dev, 51, (4, C), dt=torch.bfloat16)
    tail = X[-4:].clone()
    Y, mean, rstd = ttt.groupnorm_fwd(X, 32, eps=EPS, act=ttt.ACT_SILU)
    alone = ttt.groupnorm_fwd(tail, 32, eps=EPS, act=ttt.ACT_SILU)
    assert torch.equal(Y[-4:], alone[0]) and torch.equal(mean[-4:], alone[1])
    dX = ttt.groupnorm_bwd(X, 32, None, None, Y, mean, rstd, ttt.ACT_SILU, dX=Y)[0]
    assert torch.equal(dX[-4:], ttt.groupnorm_bwd(tail, 32, None, None, *alone, ttt.ACT_SILU)[0])
    # one long slab: its places past 2^31 elements
    S = ttt.groupnorm_fwd(X[None, :1 << 20].contiguous(), 32, eps=EPS)[0]
    assert (S == 0).all()
    del S, dX, Y
    rng = torch.tensor([3, 1 << 40], device=dev)
    Y = ttt.dropout(X, 0.5, rng)
    later = rng.clone()
    later[1] += (rows - 4) * C // 4
    assert torch.equal(Y[-4:], ttt.dropout(tail, 0.5, later))


def test_delta_past_32_bits(dev):
    """More than 2^31 elements of keys in one head: a document that starts anew near the end is what
    it is alone, and so are its gradients."""
    import torch
    T, d, dv, n = (1 << 24) + 64 + 40, 128, 16, 104
    K = torch.zeros(1, 1, T, d, dtype=torch.bfloat16, device=dev)
    V = torch.zeros(1, 1, T, dv, dtype=torch.bfloat16, device=dev)
    eta, g = torch.full((1, 1, T), 0.5, device=dev), torch.zeros(1, 1, T, device=dev)
    k, = tensors(dev, 52, (1, 1, n, d))
    K[:, :, -n:] = torch.nn.functional.normalize(k, dim=-1).bfloat16()
    V[:, :, -n:], = tensors(dev, 53, (1, 1, n, dv), dt=torch.bfloat16)
    g[:, :, -n] = -float("inf")
    Z, W = ttt.delta_fwd(K, K, V, eta, g)
    tail = [t[:, :, -n:].clone() for t in (K, K, V, eta, g)]
    z, w = ttt.delta_fwd(*tail)
    rel = ref.delta_rel(n, d, dv)
    assert (W - w).abs().max() <= 2 * rel * w.abs().max()
    # (chunks end elsewhere: two roundings to bf16 of nearly the same values)
    assert (Z[:, :, -n:].float() - z.float()).abs().max() <= (2.0 ** -8 + 2 * ref.Z_BF16) * z.float().abs().max()
    assert (Z[:, :, :-n] == 0).all()
