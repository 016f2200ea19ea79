"""The group norm's form for large groups (past 4096 vectors, the places shared out over workgroups):
the properties that hold for small groups hold there, each at a shape that asks for its workspace."""
import numpy as np
import pytest

import delta_ref as ref
from test_gpu_graph import capture, eager_noise, nan_fill
from test_gpu_groupnorm import ACT, EPS, check, make, np64
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu

# N, S, C, G: two with the places in several parts, one whose rows take one part each
SHAPES = [(2, 5000, 64, 4), (3, 5000, 96, 4), (1100, 8, 4128, 1)]


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def setup(dev, shape, io, seed, **kw):
    N, S, C, G = shape
    assert ttt.groupnorm_workspace_bytes(N, S, C, G, ttt.DTYPE_BF16 if io == "bf16" else ttt.DTYPE_F32) > 0
    return make(dev, N, S, C, io, seed, **kw)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_parity_of_rows_in_one_part(dev, io, act):
    """Enough rows that no row's places are shared out: the shape's own rows, four of them checked."""
    N, S, C, G = SHAPES[2]
    X, w, b, dY = setup(dev, SHAPES[2], io, 1)
    Y, mean, rstd = ttt.groupnorm_fwd(X, G, w, b, EPS, ACT[act])
    dX = ttt.groupnorm_bwd(X, G, w, b, dY, mean, rstd, ACT[act])[0]
    rows = [0, 1, N // 2, N - 1]
    y, m, r, ey, em, er = ref.groupnorm(np64(X[rows]), G, np64(w), np64(b), EPS, act)
    assert ref.within(np64(Y[rows]), y, ey, io)[0]
    assert ref.within(np64(mean[rows]), m, em, "f32")[0] and ref.within(np64(rstd[rows]), r, er * r, "f32")[0]
    (dx, _, _), (ex, _, _) = ref.groupnorm_bwd(np64(X[rows]), G, np64(w), np64(b), np64(dY[rows]), np64(mean[rows]),
                                               np64(rstd[rows]), act)
    assert ref.within(np64(dX[rows]), dx, ex, io)[0]


@pytest.mark.parametrize("shape", SHAPES[:2])
@pytest.mark.parametrize("far", [30.0, 1000.0])
def test_far_means(dev, shape, far):
    X, w, b, dY = setup(dev, shape, "f32", 3, far=far)
    check(X, w, b, dY, shape[3], "f32", "silu")


@pytest.mark.parametrize("shape", SHAPES[:2])
def test_constant_groups(dev, shape):
    import torch
    X, w, b, dY = setup(dev, shape, "f32", 4)
    X = torch.full_like(X, 0.75)
    _, mean, _, _ = check(X, w, b, dY, shape[3], "f32", "none", 1e-3)
    assert (mean == 0.75).all()


@pytest.mark.parametrize("place", [0, 777])
def test_non_finite_values_stay_in_their_group(dev, place):
    shape = (3, 5000, 96, 4)
    X, w, b, dY = setup(dev, shape, "bf16", 5)
    N, S, C, G = shape
    clean = ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_SILU)
    grads = ttt.groupnorm_bwd(X, G, w, b, dY, *clean[1:], ttt.ACT_SILU)[0]
    X[1, place, C // G], X[2, place, 0] = float("nan"), float("inf")
    got = ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_SILU)
    back = ttt.groupnorm_bwd(X, G, w, b, dY, *got[1:], ttt.ACT_SILU)[0]
    per = C // G
    assert got[0][1, :, per:2 * per].isnan().all() and got[0][2, :, :per].isnan().any()
    for a, c in ((got[0], clean[0]), (back, grads)):
        assert (a[0] == c[0]).all() and (a[1, :, :per] == c[1, :, :per]).all()
        assert (a[1, :, 2 * per:] == c[1, :, 2 * per:]).all() and (a[2, :, per:] == c[2, :, per:]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_in_place_and_same_bits(dev, shape, io):
    X, w, b, dY = setup(dev, shape, io, 6)
    G = shape[3]
    Y, mean, rstd = ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_GELU)
    X1 = X.clone()
    assert (ttt.groupnorm_fwd(X1, G, w, b, EPS, ttt.ACT_GELU, Y=X1)[0] == Y).all()
    first = ttt.groupnorm_bwd(X, G, w, b, dY, mean, rstd, ttt.ACT_GELU)
    for place in ("X", "dY"):
        X1, dY1 = X.clone(), dY.clone()
        got = ttt.groupnorm_bwd(X1, G, w, b, dY1, mean, rstd, ttt.ACT_GELU, dX=X1 if place == "X" else dY1)
        assert all((p == q).all() for p, q in zip(got, first))


def test_outputs_end_where_they_should(dev):
    import torch
    X, w, b, dY = setup(dev, (2, 9000, 24, 3), "bf16", 8)
    n = X.numel()
    room = torch.full((n + 256,), 7.0, dtype=torch.bfloat16, device=dev)
    _, mean, rstd = ttt.groupnorm_fwd(X, 3, w, b, Y=room[:n].view(X.shape))
    assert (room[n:] == 7).all()
    wide = [torch.full((24 + 64,), 7.0, device=dev) for _ in range(2)]
    ttt.groupnorm_bwd(X, 3, w, b, dY, mean, rstd, dX=room[:n].view(X.shape), dweight=wide[0][:24], dbias=wide[1][:24])
    assert (room[n:] == 7).all() and all((t[24:] == 7).all() for t in wide)


@pytest.mark.parametrize("shape", SHAPES)
def test_graphs_replay(dev, shape):
    import torch
    N, S, C, G = shape
    X, w, b, dY = setup(dev, shape, "bf16", 9)
    byte = lambda n: torch.empty(n, dtype=torch.uint8, device=dev)  # noqa: E731
    wf, wb = byte(ttt.groupnorm_workspace_bytes(*shape, 1)), byte(ttt.groupnorm_bwd_workspace_bytes(*shape, 1))
    mean0, rstd0 = ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_GELU)[1:]
    outs = [torch.empty_like(t) for t in (X, mean0, rstd0, X, w, b)]

    def step():
        ttt.groupnorm_fwd(X, G, w, b, EPS, ttt.ACT_GELU, Y=outs[0], mean=outs[1], rstd=outs[2], workspace=wf)
        ttt.groupnorm_bwd(X, G, w, b, dY, mean0, rstd0, ttt.ACT_GELU, dX=outs[3], dweight=outs[4], dbias=outs[5],
                          workspace=wb)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    g = capture(step)
    for k in range(4):
        nan_fill(*outs)
        eager_noise(dev)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, want)), k
