"""Rows of very many features: the sums' errors do not grow with their length.

A thread adds 8 terms in fp32, those sums in fp64, and 256 threads' sums meet in 8 additions: with the
conversion a term passes through at most 17 roundings, whatever D is.  k = 1 / sqrt(mean(r^2) + eps) takes half
of that and of r's own two, of the division's and of the addition's of eps, and 4 for the reciprocal root:
REL = 0.5 (17 + 2 + 2) + 4 half-steps of fp32."""
import numpy as np
import pytest

import block_ref as ref
from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu

EPS, U = 1e-6, ref.U
SUM = 17
REL = 0.5 * (SUM + 4) + 4


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def make(dev, rows, D, io, values, seed=7):
    import torch
    gen = torch.Generator(device="cpu").manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    t = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    X, res, dY = t(rows, D), 2 * t(rows, D), t(rows, D)
    if values == "equal":       # terms of one size and sign: roundings that do not cancel
        X[:], res[:], dY[:] = 0.7, 0.3, 0.9
    return X.to(dev, dt), (1 + 0.3 * t(D)).to(dev), res.to(dev, dt), dY.to(dev, dt)


WIDE = [(3, 1 << 20, "bf16"), (2, (1 << 20) + 5, "f32"), (1, (1 << 23) + 1, "f32"), (1, 1 << 24, "bf16")]


@pytest.mark.parametrize("values", ["equal", "normal"])
@pytest.mark.parametrize("rows,D,io", WIDE)
def test_forward(dev, rows, D, io, values):
    say("case", rows, D, io, values)
    X, w, res, _ = make(dev, rows, D, io, values)
    for residual in (res, None):
        y, r = ref.rmsnorm(np64(X), np64(w), np64(residual), EPS)
        Y, R = ttt.rmsnorm_fwd(X, w, residual, EPS)
        ok, worst = ref.within(np64(Y), y, np.abs(y) * (REL + 4) * U, io)
        say("  error over what is allowed: y %.3f" % worst)
        assert ok
        Y8, scale, _ = ttt.rmsnorm_q8_fwd(X, w, residual, EPS)
        top = np.abs(y).max(-1) / ref.E4M3_MAX
        ok, worst = ref.within(np64(scale), top, top * (REL + 4) * U, "f32")
        say("  error over what is allowed: scale %.3f" % worst)
        assert ok


@pytest.mark.parametrize("values", ["equal", "normal"])
@pytest.mark.parametrize("rows,D,io", WIDE)
def test_backward(dev, rows, D, io, values):
    """m = mean(u n): SUM + 4 roundings of the mean of |u n| (the product's, r's two, the division's), and
    k's; dx = k (u - n m) + dr: three more each."""
    say("case", rows, D, io, values)
    R, w, dR, dY = make(dev, rows, D, io, values, 8)
    r, dy, weight = np64(R), np64(dY), np64(w)
    k = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + EPS)
    n, u = np.abs(r * k), np.abs(dy * weight)
    m = (u * n).mean(-1, keepdims=True)
    for extra in (dR, None):
        dx, dw = ref.rmsnorm_bwd(r, weight, dy, np64(extra), EPS)
        edx = k * (u * (REL + 6) + n * m * (3 * REL + SUM + 4 + 8)) * U
        if extra is not None:
            edx = edx + 2 * U * (np.abs(np64(extra)) + k * (u + n * m))
        edw = (rows + REL + 4) * U * (np.abs(dy) * n).sum(0)
        dX, dweight = ttt.rmsnorm_bwd(R, w, dY, extra, EPS)
        ok, worst = ref.within(np64(dX), dx, edx, io)
        ok2, worst2 = ref.within(np64(dweight), dw, edw, "f32")
        say("  error over what is allowed: dx %.3f dw %.3f" % (worst, worst2))
        assert ok and ok2


@pytest.mark.parametrize("rows,D,io", [(1500, 17000, "bf16"), (1100, 9001, "f32"), (4, 300000, "bf16"),
                                       (0, 20000, "bf16")])
def test_backward_in_place(dev, rows, D, io):
    """dX at dY's or dR's place: dweight is formed of what stood there."""
    import torch
    say("case", rows, D, io)
    R, w, dR, dY = make(dev, rows, D, io, "normal", 9)
    dX, dw = ttt.rmsnorm_bwd(R, w, dY, dR, EPS)
    r, dy = np64(R), np64(dY)
    n = r / np.sqrt((r * r).mean(-1, keepdims=True) + EPS)
    # 8 terms at a time in fp32, those sums in fp64 and rounded, up to 2^18 / 9001 = 29 planes in fp32, and
    # k's and n's own
    room = (8 + 1 + 29 + REL + 2) * U * (np.abs(dy) * np.abs(n)).sum(0)
    assert ref.within(np64(dw), (dy * n).sum(0), room, "f32")[0]
    for k in (0, 1):
        a, b = dY.clone(), dR.clone()
        _, dw2 = ttt.rmsnorm_bwd(R, w, a, b, EPS, dX=(a, b)[k])
        torch.cuda.synchronize()
        assert torch.equal((a, b)[k], dX) and torch.equal(dw, dw2)
