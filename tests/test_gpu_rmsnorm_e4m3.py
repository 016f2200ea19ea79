"""The norm's e4m3 values are those of its formula: with t = r w, the e4m3 value nearest to
448 t / max|t| (ties to even), decided in fp64.  What the kernel forms is good to a few 2^-52, and so is the
fp64 form here: they are compared for equality."""
import numpy as np
import pytest

from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def nearest(X, w, res):
    """The e4m3 values (as fp64) of every row."""
    t = X.astype(np.float64) + (0.0 if res is None else res.astype(np.float64))
    if w is not None:
        t = t * w.astype(np.float64)
    v = t * 448.0 / np.abs(t).max(-1, keepdims=True)
    # steps: three binary digits after the first, 2^-9 at the bottom
    step = np.ldexp(1.0, np.maximum(np.frexp(v)[1] - 1, -6) - 3)
    return np.round(v / step) * step


def check(dev, X, w, res, io):
    """X, res: fp32 arrays that the type holds; w: fp32 or None."""
    import torch
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    on = lambda a: None if a is None else torch.from_numpy(a).to(dev, dt)  # noqa: E731
    for row in (X, res):
        assert row is None or np.array_equal(torch.from_numpy(row).to(dt).float().numpy(), row)
    weight, x, z = None if w is None else torch.from_numpy(w).to(dev), on(X), on(res)
    Y8, scale, R = ttt.rmsnorm_q8_fwd(x, weight, z, EPS, R=torch.empty_like(x))
    # r at an input's place: what is read a second time is read before it is written
    a, b = x.clone(), None if z is None else z.clone()
    for at in (a,) if b is None else (b, a):
        Z8, scale2, _ = ttt.rmsnorm_q8_fwd(a, weight, b if at is b else z, EPS, R=at)
        assert torch.equal(Z8.view(torch.uint8), Y8.view(torch.uint8)) and torch.equal(scale2, scale)
        assert torch.equal(at, R)
    got, want = Y8.float().cpu().numpy().astype(np.float64), nearest(X, w, res)
    off = int((got != want).sum())
    say("  %d of %d values differ" % (off, want.size))
    assert off == 0


def in_type(a, io):
    import torch
    t = torch.from_numpy(np.asarray(a, np.float32))
    return (t.to(torch.bfloat16) if io == "bf16" else t).float().numpy()


# midpoints of neighbouring e4m3 values, from the largest down to the bottom's
TIES = np.array([432, 400, 17, 19, 15.5, 1.0625, 2.0 ** -6 * 1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 100, 232])


@pytest.mark.parametrize("D", [33, 34, 67, 200, 777, 2048, 5001, 20000])
@pytest.mark.parametrize("weight", [False, True])
def test_next_to_a_tie(dev, D, weight):
    """fp32 values at the places where two e4m3 values meet, and one fp32 step to either side of them."""
    say("case D", D, "weight", weight)
    gen = np.random.default_rng(D)
    most = gen.uniform(1.0, 2.0, 64).astype(np.float32)
    w = gen.uniform(0.5, 2.0, D).astype(np.float32) if weight else None
    by = np.ones(D) if w is None else w.astype(np.float64)
    top = most * by[0]
    X = np.empty((64, D), np.float32)
    for c in range(1, D):
        at = (TIES[c % len(TIES)] / 448.0 * top / by[c]).astype(np.float32)
        X[:, c] = (at, np.nextafter(at, np.float32(9e9)), np.nextafter(at, np.float32(0)), -at)[c % 4]
    X[:, 0] = most
    check(dev, X, w, None, "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [33, 300, 4100])
def test_ties_go_to_even(dev, D, io):
    """Values whose quotient is a midpoint exactly, at several powers of two."""
    X = np.empty((12, D), np.float32)
    for k in range(12):
        X[k] = np.ldexp(np.resize(np.concatenate([TIES, -TIES, [448.0, 3.0, 0.0]]), D), k - 6)
        X[k, 5] = np.ldexp(448.0, k - 6)
    check(dev, in_type(X, io), None, None, io)


@pytest.mark.parametrize("rows,D,io", [(4000, 64, "bf16"), (1000, 768, "bf16"), (2000, 2048, "bf16"),
                                       (500, 8192, "bf16"), (100, 20000, "bf16"), (60, 40000, "bf16"),
                                       (2000, 100, "f32"), (1000, 1537, "f32"), (300, 9000, "f32"),
                                       (100, 20000, "f32")])
def test_ordinary_rows(dev, rows, D, io):
    say("case", rows, D, io)
    gen = np.random.default_rng(rows + D)
    X, res = (in_type(s * gen.standard_normal((rows, D)), io) for s in (1.0, 2.0))
    w = (1 + 0.3 * gen.standard_normal(D)).astype(np.float32)
    check(dev, X, w, res, io)
    check(dev, X, w, None, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [33, 64, 1024, 5000, 40000])
def test_a_weight_that_is_not_finite(dev, D, io):
    """A NaN weight makes every row's scale and values NaN; an infinite one (the largest |y| is infinite)
    the values, and the scale infinite."""
    import torch
    X = torch.from_numpy(in_type(np.random.default_rng(D).standard_normal((5, D)), io)).to(dev)
    X = X.to(torch.bfloat16 if io == "bf16" else torch.float32)
    for bad in (float("nan"), float("inf")):
        for at in (D // 2, D - 1):
            w = torch.ones(D, device=dev)
            w[at] = bad
            Y8, scale, _ = ttt.rmsnorm_q8_fwd(X, w, None, EPS)
            assert torch.isnan(Y8.float()).all()
            assert (torch.isnan(scale) if bad != bad else torch.isposinf(scale)).all()
