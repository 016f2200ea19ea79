"""GPU parity of the group norm with an activation (forward, backward) with its fp64 form, within
the bounds that delta_ref derives."""
import numpy as np
import pytest

import delta_ref as ref
from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu

EPS = 1e-5
ACT = {"none": ttt.ACT_NONE, "silu": ttt.ACT_SILU, "gelu": ttt.ACT_GELU}


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def make(dev, N, S, C, io, seed, affine=True, far=0.0):
    import torch
    gen = torch.Generator(device="cpu").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    X = (n(N, S, C) * (0.5 + torch.rand(C, generator=gen)) + 0.5 * n(C) + far).to(dt).to(dev)
    return (X, (1 + 0.3 * n(C)).to(dev) if affine else None, (0.3 * n(C)).to(dev) if affine else None,
            n(N, S, C).to(dt).to(dev))


def check(X, w, b, dY, G, io, act, eps=EPS):
    Y, mean, rstd = ttt.groupnorm_fwd(X, G, w, b, eps, ACT[act])
    y, m, r, ey, em, er = ref.groupnorm(np64(X), G, np64(w), np64(b), eps, act)
    for name, got, want, bound, t in (("y", Y, y, ey, io), ("mean", mean, m, em, "f32"), ("rstd", rstd, r, er * r, "f32")):
        ok, worst = ref.within(np64(got), want, bound, t)
        say("  %s: error over what is allowed %.3f" % (name, worst))
        assert ok, name
    got = ttt.groupnorm_bwd(X, G, w, b, dY, mean, rstd, ACT[act])
    want, bound = ref.groupnorm_bwd(np64(X), G, np64(w), np64(b), np64(dY), np64(mean), np64(rstd), act)
    for name, a, c, e, t in zip(("dx", "dweight", "dbias"), got, want, bound, (io, "f32", "f32")):
        if a is None:
            assert w is None
            continue
        ok, worst = ref.within(np64(a), c, e, t)
        say("  %s: error over what is allowed %.3f" % (name, worst))
        assert ok, name
    return Y, mean, rstd, got


SHAPES = [
    # N, S, C, G
    (1, 1, 64, 1), (5, 1, 64, 8), (7, 1, 24, 8), (3, 1, 3, 1), (9, 1, 20, 1), (1000, 1, 96, 32), (4, 1, 2048, 32),
    (3, 1, 4096, 4), (2, 1, 640, 1), (600, 1, 160, 2), (2, 1, 5000, 1), (2, 49, 24, 8), (1, 100, 64, 4), (2, 1000, 640, 32),
    (3, 2, 7, 7), (1, 5000, 5, 1), (40, 2, 512, 8), (30, 1, 4096, 1), (3, 1, 65536, 1), (2, 8, 8192, 2), (4, 3, 1200, 5),
    (1, 40000, 6, 2), (2, 300, 4096, 32), (70, 9, 32, 4), (1, 33, 2051, 7),
]


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_parity(dev, shape, io, act):
    N, S, C, G = shape
    X, w, b, dY = make(dev, N, S, C, io, sum(shape), affine=(N + S) % 4 != 0)
    check(X, w, b, dY, G, io, act)


@pytest.mark.parametrize("shape", [(6, 1, 256, 4), (2, 700, 64, 4)])
def test_far_means(dev, shape):
    """Means a thousand times the spread: sums of squares would lose it."""
    N, S, C, G = shape
    X, w, b, dY = make(dev, N, S, C, "f32", 3, far=1000.0)
    check(X, w, b, dY, G, "f32", "silu")


@pytest.mark.parametrize("shape", [(6, 1, 256, 4), (2, 700, 64, 4)])
def test_constant_groups(dev, shape):
    import torch
    N, S, C, G = shape
    X, w, b, dY = make(dev, N, S, C, "f32", 4)
    X = torch.full_like(X, 0.75)
    Y, mean, rstd, _ = check(X, w, b, dY, G, "f32", "none", 1e-3)
    assert (mean == 0.75).all()


@pytest.mark.parametrize("shape", [(6, 1, 256, 4), (3, 700, 64, 4)])
def test_non_finite_values_stay_in_their_group(dev, shape):
    N, S, C, G = shape
    X, w, b, dY = make(dev, N, S, C, "bf16", 5)
    clean = ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_SILU)[0]
    X[1, 0, C // G] = float("nan")
    X[2, 0, 0] = float("inf")
    Y = ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_SILU)[0]
    per = C // G
    assert Y[1, :, per:2 * per].isnan().all() and Y[2, :, :per].isnan().any()
    assert (Y[0] == clean[0]).all() and (Y[1, :, :per] == clean[1, :, :per]).all()
    assert (Y[1, :, 2 * per:] == clean[1, :, 2 * per:]).all() and (Y[2, :, per:] == clean[2, :, per:]).all()


@pytest.mark.parametrize("shape", [(60, 1, 256, 4), (2, 700, 64, 4)])
def test_in_place_and_same_bits(dev, shape):
    N, S, C, G = shape
    X, w, b, dY = make(dev, N, S, C, "bf16", 6)
    Y, mean, rstd = ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_GELU)
    X1 = X.clone()
    assert (ttt.groupnorm_fwd(X1, G, w, b, EPS, ttt.ACT_GELU, Y=X1)[0] == Y).all()
    first = ttt.groupnorm_bwd(X, G, w, b, dY, mean, rstd, ttt.ACT_GELU)
    for place in ("X", "dY"):
        X1, dY1 = X.clone(), dY.clone()
        got = ttt.groupnorm_bwd(X1, G, w, b, dY1, mean, rstd, ttt.ACT_GELU, dX=X1 if place == "X" else dY1)
        assert all((p == q).all() for p, q in zip(got, first))


def test_shapes_with_several_axes(dev):
    X, w, b, dY = make(dev, 2, 12, 32, "f32", 7)
    a = ttt.groupnorm_fwd(X, 4, w, b)
    c = ttt.groupnorm_fwd(X.view(2, 3, 4, 32), 4, w, b)
    assert all((p.reshape(-1) == q.reshape(-1)).all() for p, q in zip(a, c)) and c[0].shape == (2, 3, 4, 32)
    assert ttt.groupnorm_fwd(X.view(24, 32), 4)[1].shape == (24, 4)


def test_nothing(dev):
    import torch
    w = torch.ones(32, device=dev)
    X = torch.empty(0, 5, 32, device=dev)
    Y, mean, rstd = ttt.groupnorm_fwd(X, 4, w, w)
    dX, dw, db = ttt.groupnorm_bwd(X, 4, w, w, X, mean, rstd)
    assert Y.numel() == 0 and (dw == 0).all() and (db == 0).all()


def test_outputs_end_where_they_should(dev):
    import torch
    for N, S, C, G in ((5, 1, 24, 8), (2, 50, 24, 8)):
        X, w, b, dY = make(dev, N, S, C, "bf16", 8)
        n = X.numel()
        room = torch.full((n + 256,), 7.0, dtype=torch.bfloat16, device=dev)
        _, mean, rstd = ttt.groupnorm_fwd(X, G, w, b, Y=room[:n].view(X.shape))
        assert (room[n:] == 7).all()
        wide = [torch.full((C + 64,), 7.0, device=dev) for _ in range(2)]
        ttt.groupnorm_bwd(X, G, w, b, dY, mean, rstd, dX=room[:n].view(X.shape), dweight=wide[0][:C], dbias=wide[1][:C])
        assert (room[n:] == 7).all() and all((t[C:] == 7).all() for t in wide)


@pytest.mark.parametrize("shape", [(70000, 1, 32, 4), (9, 3, 40, 5), (2, 9000, 40, 5)])
def test_weight_or_bias_alone(dev, shape):
    N, S, C, G = shape
    X, w, b, dY = make(dev, N, S, C, "f32", 9)
    for ww, bb in ((w, None), (None, b)):
        Y, mean, rstd = ttt.groupnorm_fwd(X, G, ww, bb, EPS, ttt.ACT_SILU)
        y, _, _, ey, _, _ = ref.groupnorm(np64(X), G, np64(ww), np64(bb), EPS, "silu")
        assert ref.within(np64(Y), y, ey, "f32")[0]
        dx, dw, db = ttt.groupnorm_bwd(X, G, ww, bb, dY, mean, rstd, ttt.ACT_SILU)
        assert (dw is None) == (ww is None) and (db is None) == (bb is None)
        want, bound = ref.groupnorm_bwd(np64(X), G, np64(ww), np64(bb), np64(dY), np64(mean), np64(rstd), "silu")
        for got, v, e in zip((dx, dw, db), want, bound):
            assert got is None or ref.within(np64(got), v, e, "f32")[0]


def test_refuses_what_does_not_fit(dev):
    import torch
    X, w, b, dY = make(dev, 4, 10, 32, "f32", 10)
    stats = torch.zeros(4, 8, device=dev)
    for call in (lambda: ttt.groupnorm_fwd(X, 5), lambda: ttt.groupnorm_fwd(X, 0), lambda: ttt.groupnorm_fwd(X[0, 0], 4),
                 lambda: ttt.groupnorm_fwd(X, 4, w[:16]), lambda: ttt.groupnorm_fwd(X, 4, w.double()),
                 lambda: ttt.groupnorm_fwd(X.transpose(1, 2), 4), lambda: ttt.groupnorm_fwd(X, 4, mean=stats),
                 lambda: ttt.groupnorm_bwd(X, 4, w, b, dY, stats, stats), lambda: ttt.groupnorm_fwd(X.cpu(), 4)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ttt.groupnorm_fwd(X.half(), 4)
