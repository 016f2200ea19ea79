"""GPU dropout against the generator's plain form: the same elements dropped, the kept ones to a
rounding."""
import numpy as np
import pytest

import delta_ref as ref
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def make(dev, n, io, seed, first):
    import torch
    gen = torch.Generator(device="cpu").manual_seed(n)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    X, R = (torch.randn(n, generator=gen).to(dt).to(dev) for _ in range(2))
    return X, R, torch.tensor([seed, first], dtype=torch.int64, device=dev)


def check(X, R, Y, n, io, p, seed, first):
    x = X.double().cpu().numpy()
    keep = ref.keep_mask(n, p, seed % (1 << 64), first % (1 << 64))
    kept = np.where(keep, x / (1 - p), 0.0)
    want = kept + (R.double().cpu().numpy() if R is not None else 0.0)
    # the scale's rounding, the product's and the sum's
    ok, worst = ref.within(Y.double().cpu().numpy(), want, 2 * ref.U * np.abs(kept) + ref.U * np.abs(want), io)
    assert ok, worst
    if R is None:
        assert ((Y.double().cpu().numpy() == 0) == (~keep | (x == 0))).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 4, 7, 8, 9, 1000, 65536, 100003])
def test_parity(dev, n, io, residual):
    for p, seed, first in ((0.1, 42, 0), (0.5, -3, 4294967290), (0.0, 1, 2), (0.9, 1 << 62, -5), (0.25, 7, (1 << 63) - 2)):
        X, R, rng = make(dev, n, io, seed, first)
        R = R if residual else None
        check(X, R, ttt.dropout(X, p, rng, R), n, io, p, seed, first)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradient_is_the_same_call(dev, io):
    X, R, rng = make(dev, 1001, io, 5, 9)
    Y = ttt.dropout(X, 0.5, rng)
    dX = ttt.dropout(R, 0.5, rng)
    # scale 2: exact in both types
    assert ((dX != 0) == ((Y != 0) & (R != 0))).all() and (dX[dX != 0] == 2 * R[dX != 0]).all()


def test_in_place(dev):
    X, R, rng = make(dev, 5000, "bf16", 5, 9)
    want = ttt.dropout(X, 0.3, rng, R)
    x, r = X.clone(), R.clone()
    assert (ttt.dropout(x, 0.3, rng, R, Y=x) == want).all()
    assert (ttt.dropout(X, 0.3, rng, r, Y=r) == want).all()


def test_dropped_values_leave_nothing(dev):
    X, R, rng = make(dev, 4096, "f32", 5, 9)
    gone = ttt.dropout(X, 0.5, rng) == 0
    X[gone] = float("nan")
    Y = ttt.dropout(X, 0.5, rng)
    assert not Y.isnan().any() and (Y[gone] == 0).all()


def test_calls_one_after_the_other_continue(dev):
    """A tensor in two calls, the second with the counter advanced, is the tensor in one."""
    import torch
    X, _, rng = make(dev, 3000, "f32", 5, 100)
    whole = ttt.dropout(X, 0.4, rng)
    a = ttt.dropout(X[:1000].contiguous(), 0.4, rng)
    rng[1] += (1000 + 3) // 4
    b = ttt.dropout(X[1000:].contiguous(), 0.4, rng)
    assert (torch.cat([a, b]) == whole).all()


def test_output_ends_where_it_should(dev):
    import torch
    for n in (5, 1003):
        X, _, rng = make(dev, n, "bf16", 5, 9)
        room = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device=dev)
        ttt.dropout(X, 0.5, rng, Y=room[:n])
        assert (room[n:] == 7).all()
