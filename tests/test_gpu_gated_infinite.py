"""Infinite and very large states under gates whose exponential, or whose product over a few tokens, is 0 in
fp32: an infinite state stays infinite up to the next reset, a finite one is forgotten, and forward, step and
backward pass agree on it wherever their runs and tiles begin.

Under such gates the formula leaves x_t of every finite state (what is left of the one before is under
2e-22 of it and x_t is no smaller than 1e-4), so the forward results are compared for equality."""
import numpy as np
import pytest

from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def left(g, h):
    """What a token's gate leaves of h, in fp64."""
    shut = np.isneginf(g)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(shut, 0.0, np.where(np.isinf(h), h, np.exp(g) * h))


def serial(g, x, h):
    """All states [N, T, d], each rounded to fp32 (so that it overflows where fp32 does)."""
    out = np.empty_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(x.shape[1]):
            h = (left(g[:, t], h) + x[:, t]).astype(np.float32).astype(np.float64)
            out[:, t] = h
    return out


def make(dev, T, d, io, gate, seed):
    """One row; channels 0 to 6 hold what the file's first lines name, the others are ordinary."""
    import torch
    gen = np.random.default_rng(seed)
    x = gen.standard_normal((1, T, d))
    x = np.where(np.abs(x) < 1e-4, 0.5, x)
    g = np.full((1, T, d), gate)
    h = gen.standard_normal((1, d))
    at = T // 3
    h[0, 0], h[0, 1] = INF, -INF
    h[0, 2] = 1e38 if gate <= -200 else 1.0
    x[0, at, 3] = INF
    x[0, at, 4], g[0, min(T - 1, at + 40), 4] = -INF, -INF          # up to a reset
    h[0, 5], x[0, at, 5] = INF, -INF                                # NaN from there on
    x[0, at:at + 2, 6], g[0, at + 1:at + 2, 6] = 3e38, 0.0          # a sum that overflows
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    X, G = (torch.from_numpy(a.astype(np.float32))[None].to(dev, dt) for a in (x, g))
    return X, G, torch.from_numpy(h.astype(np.float32))[None].to(dev)


def np64(t):
    return t.double().cpu().numpy()[0]


def rounded(a, io):
    import torch
    with np.errstate(over="ignore"):
        t = torch.from_numpy(a.astype(np.float32))
    return (t.to(torch.bfloat16) if io == "bf16" else t).double().numpy()


def same(a, b):
    return np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.nan_to_num(a, nan=0.0, posinf=INF, neginf=-INF),
                                                                       np.nan_to_num(b, nan=0.0, posinf=INF, neginf=-INF))


GATES = [-50.0, -200.0, -1e4]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,d", [(3, 64), (12, 83), (60, 64), (700, 83), (5000, 64), (5000, 16), (3000, 520)])
def test_forward_and_step(dev, T, d, io, gate):
    import torch
    say("case", T, d, io, gate)
    X, G, h0 = make(dev, T, d, io, gate, T + d)
    want = serial(np64(G), np64(X), np64(h0))
    Z, hT = ttt.gated_fwd(X, G, h0)
    assert same(np64(Z), rounded(want, io)) and same(np64(hT), want[:, -1])
    h, Zs, t = h0.clone(), [], 0
    for n in (1, 1, 5, T):
        n = min(n, T - t)
        if n > 0:
            Zs.append(ttt.gated_step(X[:, :, t:t + n].clone(), G[:, :, t:t + n].clone(), h))
            t += n
    assert same(np64(torch.cat(Zs, 2)), rounded(want, io)) and same(np64(h), want[:, -1])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,d", [(3, 64), (60, 64), (700, 83), (5000, 64), (3000, 520)])
def test_backward(dev, T, d, io, gate):
    """dX is the same recurrence from the other end; dG = exp(g) lambda h and dh0 have products below
    fp32's range (2^-126, taken as 0), one exponential (2 half-steps and 3 |g| of them) and three
    roundings, the reference's own among them."""
    say("case", T, d, io, gate)
    dZ, G, dh = make(dev, T, d, io, gate, T + d + 1)
    dZ, G = dZ.flip(2).contiguous(), G.flip(2).contiguous()
    Z = make(dev, T, d, io, gate, 5)[0].nan_to_num(1.0, 1.0, 1.0).clamp(-4, 4)
    h0 = make(dev, T, d, io, gate, 6)[2].clamp(-4, 4)
    g, z, dz = np64(G), np64(Z), np64(dZ)
    after = np.concatenate([g[:, 1:], np.zeros_like(g[:, :1])], 1)
    lam = serial(after[:, ::-1], dz[:, ::-1], np64(dh))[:, ::-1]
    dX, dG, dh0 = ttt.gated_bwd(G, Z, dZ, h0, dh)
    if gate <= -200:             # the last token's lambda is dz + dh: the only sum
        assert same(np64(dX), rounded(lam, io))
    before = np.concatenate([np64(h0)[:, None], z[:, :-1]], 1)
    back = left(g, lam)
    with np.errstate(invalid="ignore", over="ignore"):      # (3e38 times -1.7 leaves fp32's range)
        want = np.where(np.isneginf(g), 0.0, back * before).astype(np.float32).astype(np.float64)
    for got, ref, half in ((np64(dG), want, 2.0 ** -8 if io == "bf16" else 2.0 ** -24),
                           (np64(dh0), back[:, 0], 2.0 ** -24)):
        fine = np.isfinite(ref)
        assert same(np.where(fine, 0.0, got), np.where(fine, 0.0, ref))
        room = np.abs(ref) * (half + (6 + 3 * abs(gate)) * 2.0 ** -24) * 1.01 + 2.0 ** -126 * 8
        assert (np.abs(got[fine] - ref[fine]) <= room[fine]).all()
