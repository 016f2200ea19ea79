"""Group norms of so many groups that a launch of their workgroups side by side would have 2^32 threads
or more, or that its grid goes on along another axis."""
import numpy as np
import pytest

import delta_ref as ref
from gpu_helpers import say
from test_gpu_groupnorm import ACT, EPS, np64
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu

X22 = 1 << 22        # workgroups along a grid's first axis


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def near(X, w, b, dY, G, act, rows, got):
    """The rows' outputs against the fp64 form; X and dY hold the rows alone."""
    Y, mean, rstd, dX = (np64(t) for t in got)
    y, m, r, ey, em, er = ref.groupnorm(X, G, w, b, EPS, act)
    (dx, _, _), (ex, _, _) = ref.groupnorm_bwd(X, G, w, b, dY, mean, rstd, act)
    for name, a, c, e, t in (("y", Y, y, ey, "bf16"), ("mean", mean, m, em, "f32"), ("rstd", rstd, r, er * r, "f32"),
                             ("dx", dX, dx, ex, "bf16")):
        ok, worst = ref.within(a, c, e, t)
        say("  %s: error over what is allowed %.3f" % (name, worst))
        assert ok, (name, rows)


# N, S, C, G, row of the first workgroup past 2^22 along x
SHAPES = [
    ((1 << 23) + 3, 2, 32, 32, 1 << 21),         # 16 threads a group: 2^24 + 6 workgroups of 256
    (4 * X22 + 5, 65, 1, 1, 4 * X22),            # 64
    (X22 + 5, 513, 1, 1, X22),                   # 256
    (X22 + 5, 2049, 1, 1, X22),                  # 512
    (X22 + 3, 4097, 1, 1, X22),                  # slabs
    (986900, 1, 4097, 1, X22 // 17),             # slabs, 17 workgroups a row: 2^24 + 84 in all
]


@pytest.mark.parametrize("shape", SHAPES)
def test_rows_on_either_side(dev, shape):
    import torch
    N, S, C, G, edge = shape
    gen = torch.Generator(device=dev).manual_seed(N)
    X = torch.empty(N, S, C, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    dY = torch.randint(-1, 2, X.shape, dtype=torch.int8, device=dev, generator=gen).to(torch.bfloat16)
    w, b = 1 + 0.1 * torch.randn(C, device=dev, generator=gen), 0.1 * torch.randn(C, device=dev, generator=gen)
    sums = sum(part.sum((0, 1), dtype=torch.float32).double() for part in dY.split(1 << 20))
    rows = sorted({0, 1, edge - 1, edge, edge + 1, 2 * edge % N, N // 2, N - 2, N - 1})
    mean, rstd = (torch.full((N, G), float("nan"), device=dev) for _ in range(2))
    act = "none"
    Y = ttt.groupnorm_fwd(X, G, w, b, EPS, ACT[act], mean=mean, rstd=rstd)[0]
    y = Y[rows].clone()
    assert mean.isfinite().all() and rstd.isfinite().all()
    del Y
    before = np64(dY[rows])
    dX, dw, db = ttt.groupnorm_bwd(X, G, w, b, dY, mean, rstd, ACT[act], dX=dY)
    near(np64(X[rows]), np64(w), np64(b), before, G, act, rows, (y, mean[rows], rstd[rows], dX[rows]))
    assert dw.isfinite().all()
    # sums of -1, 0 and 1: exact up to 2^24 in a thread's fp32 and behind it in fp64, rounded once
    assert ((db.double() - sums).abs() <= ref.U * sums.abs()).all()
