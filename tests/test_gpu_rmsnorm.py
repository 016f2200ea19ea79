"""GPU parity of the RMS norm with residual (I/O type and e4m3 outputs, backward) with its fp64
form, within the bounds that block_ref derives."""
import numpy as np
import pytest

import block_ref as ref
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


def make(dev, rows, D, io, seed):
    import torch
    gen = torch.Generator(device="cpu").manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    t = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return (t(rows, D).to(dev, dt), (1 + 0.3 * t(D)).to(dev), (2 * t(rows, D)).to(dev, dt),
            t(rows, D).to(dev, dt))


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def check_fwd(X, w, res, Y, R, io):
    y, r = ref.rmsnorm(np64(X), np64(w), np64(res), EPS)
    D = X.shape[-1]
    ok, worst = ref.within(np64(Y), y, np.abs(y) * (ref.rms_rel(D) + 4) * ref.U, io)
    say("  error over what is allowed: y %.3f" % worst)
    assert ok
    if R is not None:
        assert ref.within(np64(R), r, np.abs(r) * ref.U, io)[0]


def check_q8(X, w, res, Y8, scale, R, io):
    y, r = ref.rmsnorm(np64(X), np64(w), np64(res), EPS)
    D = X.shape[-1]
    c = (ref.rms_rel(D) + 8) * ref.U
    sc = np.abs(y).max(-1) / ref.E4M3_MAX
    got = np64(scale)
    assert ref.within(got, sc, sc * c, "f32")[0]
    # one rounding to e4m3: half a step is 2^-4 of the value, or 2^-10 scales at the bottom
    q = np64(Y8.float())
    err = np.abs(q * got[..., None] - y)
    room = np.maximum(np.abs(y) * 2.0 ** -4, got[..., None] * 2.0 ** -10) * (1 + 4 * c) + 2 * c * np.abs(y)
    # (denormal numbers: half a step of a scale, 2^-150, times up to 448, and half a step of y)
    room = room + 449 * 2.0 ** -150
    say("  error over what is allowed: q %.3f" % float((err / np.maximum(room, 1e-300)).max()))
    assert (err <= room).all()
    live = sc > 0
    assert (np.abs(q).max(-1)[live] == ref.E4M3_MAX).all() and (q[~live] == 0).all()
    if R is not None:
        assert ref.within(np64(R), r, np.abs(r) * ref.U, io)[0]


def check_bwd(R, w, dY, dR, dX, dw, io):
    args = (np64(R), np64(w), np64(dY), np64(dR), EPS)
    want, bound = ref.rmsnorm_bwd(*args), ref.rmsnorm_bwd_bound(*args)
    ok, worst = ref.within(np64(dX), want[0], bound[0], io)
    ok2, worst2 = ref.within(np64(dw), want[1], bound[1], "f32")
    say("  error over what is allowed: dx %.3f dw %.3f" % (worst, worst2))
    assert ok and ok2


WIDTHS = [1, 2, 7, 8, 16, 33, 64, 65, 100, 128, 256, 500, 512, 513, 768, 1000, 1024, 1537, 2048, 4096,
          4100, 8192, 10007, 16384, 20000]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(dev, D, io):
    say("case D", D, io)
    for rows in (1, 37):
        X, w, res, dY = make(dev, rows, D, io, D + rows)
        for weight, residual in ((w, res), (None, None), (w, None)):
            Y, R = ttt.rmsnorm_fwd(X, weight, residual, EPS)
            check_fwd(X, weight, residual, Y, R, io)
            assert (R is None) == (residual is None)
            Y8, scale, R = ttt.rmsnorm_q8_fwd(X, weight, residual, EPS)
            check_q8(X, weight, residual, Y8, scale, R, io)
            dX, dw = ttt.rmsnorm_bwd(X, weight, dY, residual, EPS)
            check_bwd(X, weight, dY, residual, dX, dw, io)


@pytest.mark.parametrize("rows", [2, 3, 63, 64, 65, 255, 257, 1000, 4099, 40001])
@pytest.mark.parametrize("D", [64, 100, 768])
def test_row_counts(dev, rows, D):
    say("case rows", rows, D)
    X, w, res, dY = make(dev, rows, D, "bf16", rows)
    Y, R = ttt.rmsnorm_fwd(X, w, res, EPS)
    check_fwd(X, w, res, Y, R, "bf16")
    Y8, scale, R = ttt.rmsnorm_q8_fwd(X, w, res, EPS)
    check_q8(X, w, res, Y8, scale, R, "bf16")
    dX, dw = ttt.rmsnorm_bwd(X, w, dY, res, EPS)
    check_bwd(X, w, dY, res, dX, dw, "bf16")


def test_head_rows_and_shapes(dev):
    """The norm of every head's row of a scan's output: [B, H, T, d] as it stands."""
    import torch
    X, w, res, dY = make(dev, 2 * 3 * 50, 64, "bf16", 5)
    Y, _ = ttt.rmsnorm_fwd(X.view(2, 3, 50, 64), w, None, EPS)
    Y2, _ = ttt.rmsnorm_fwd(X, w, None, EPS)
    Y8, scale, _ = ttt.rmsnorm_q8_fwd(X.view(2, 3, 50, 64), w, None, EPS)
    dX, _ = ttt.rmsnorm_bwd(X.view(2, 3, 50, 64), w, dY.view(2, 3, 50, 64), None, EPS)
    assert Y.shape == (2, 3, 50, 64) and scale.shape == (2, 3, 50) and dX.shape == Y.shape
    assert torch.equal(Y.view(-1, 64), Y2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 100, 2048])
def test_in_place(dev, io, D):
    """Y at X, R at residual or X; dX at dY or dR."""
    import torch
    X, w, res, dY = make(dev, 50, D, io, 9)
    Y, R = ttt.rmsnorm_fwd(X, w, res, EPS)
    a, b = X.clone(), res.clone()
    ttt.rmsnorm_fwd(a, w, b, EPS, Y=a, R=b)
    assert torch.equal(a, Y) and torch.equal(b, R)
    a = X.clone()
    Y2, _ = ttt.rmsnorm_fwd(a, w, res, EPS, R=a)
    assert torch.equal(a, R) and torch.equal(Y2, Y)
    Y8, scale, _ = ttt.rmsnorm_q8_fwd(X, w, res, EPS)
    b = res.clone()
    Z8, scale2, _ = ttt.rmsnorm_q8_fwd(X, w, b, EPS, R=b)
    assert torch.equal(Y8.view(torch.uint8), Z8.view(torch.uint8)) and torch.equal(scale, scale2)
    assert torch.equal(b, R)
    dX, dw = ttt.rmsnorm_bwd(X, w, dY, res, EPS)
    for k in (0, 1):
        a, b = dY.clone(), res.clone()
        _, dw2 = ttt.rmsnorm_bwd(X, w, a, b, EPS, dX=(a, b)[k])
        assert torch.equal((a, b)[k], dX) and torch.equal(dw2, dw)
    dX2, none = ttt.rmsnorm_bwd(X, w, dY, res, EPS, want_dweight=False)
    assert none is None and torch.equal(dX2, dX)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 100, 2048])
def test_rows_of_zeros_and_what_is_not_finite(dev, io, D):
    """A row of zeros, and rows with an infinity or a NaN, next to ordinary ones."""
    import torch
    X, w, res, dY = make(dev, 9, D, io, 11)
    X[2] = 0
    X[4, D // 2] = float("inf")
    X[6, 1] = float("nan")
    Y, R = ttt.rmsnorm_fwd(X, w, None, EPS, R=torch.empty_like(X))
    Y8, scale, _ = ttt.rmsnorm_q8_fwd(X, w, None, EPS)
    dX, dw = ttt.rmsnorm_bwd(X, w, dY, None, EPS)
    assert torch.equal(R.nan_to_num(7.0), X.nan_to_num(7.0))
    assert (Y[2] == 0).all() and (Y8[2].float() == 0).all() and scale[2] == 0
    assert torch.isnan(scale[4]) and torch.isnan(scale[6])
    assert torch.isnan(Y8[4].float()).all() and torch.isnan(Y8[6].float()).all()
    assert torch.isnan(Y[4, D // 2]) and torch.isnan(Y[6]).all()
    assert torch.isnan(dX[6]).all()
    keep = [0, 1, 2, 3, 5, 7, 8]
    check_fwd(X[keep], w, None, Y[keep], R[keep], io)
    check_q8(X[keep], w, None, Y8[keep], scale[keep], None, io)
    want, bound = (f(np64(X[keep]), np64(w), np64(dY[keep]), None, EPS)
                   for f in (ref.rmsnorm_bwd, ref.rmsnorm_bwd_bound))
    assert ref.within(np64(dX[keep]), want[0], bound[0], io)[0]


def test_small_and_large_values(dev):
    """Rows whose values are far from 1, down to where eps decides."""
    X, w, res, dY = make(dev, 8, 300, "f32", 13)
    for k in range(8):
        X[k] *= 10.0 ** (2 * k - 8)
    Y, _ = ttt.rmsnorm_fwd(X, w, None, EPS)
    check_fwd(X, w, None, Y, None, "f32")
    Y8, scale, _ = ttt.rmsnorm_q8_fwd(X, w, None, EPS)
    check_q8(X, w, None, Y8, scale, None, "f32")
    dX, dw = ttt.rmsnorm_bwd(X, w, dY, None, EPS)
    check_bwd(X, w, dY, None, dX, dw, "f32")


@pytest.mark.parametrize("D", [3, 64, 300, 70000])
def test_e4m3_at_the_ends_of_fp32(dev, D):
    """Rows and weights whose products, or whose reciprocals, leave fp32's range; a row so small that
    its scale is 0."""
    import torch
    X, w, res, dY = make(dev, 6, D, "f32", 23)
    X[0] *= 1e-36
    X[1] *= 1e-31
    X[2] *= 1e15
    for far in (1.0, 1e17, 1e-10):
        weight = w * far
        Y8, scale, _ = ttt.rmsnorm_q8_fwd(X, weight, None, EPS)
        check_q8(X[1:], weight, None, Y8[1:], scale[1:], None, "f32")
        assert torch.isfinite(Y8[0].float()).all()
        y, _ = ref.rmsnorm(np64(X), np64(weight), None, EPS)
        err = np.abs(np64(Y8[0].float()) * np64(scale[0]) - y[0])
        # half an e4m3 step is 2^-4 of the value down to 2^-6 of the scale and, as the steps stay 2^-9
        # below that, 2^-10 of the scale at the bottom (70000 columns have values there); half a step
        # of a scale that is a denormal number is 2^-150, times up to 448
        room = np.maximum(np.abs(y[0]) * 2.0 ** -4, np64(scale[0]) * 2.0 ** -10) * 1.001
        assert (err <= room + 449 * 2.0 ** -150).all()
    X[0] *= 1e-9
    Y8, scale, _ = ttt.rmsnorm_q8_fwd(X, w * 1e-10, None, EPS)
    assert scale[0] == 0 and (Y8[0].float() == 0).all()


def test_no_rows(dev):
    import torch
    X = torch.empty(0, 64, dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    assert ttt.rmsnorm_fwd(X, w)[0].shape == (0, 64)
    assert ttt.rmsnorm_q8_fwd(X, w)[1].shape == (0,)
    dX, dw = ttt.rmsnorm_bwd(X, w, X)
    torch.cuda.synchronize()
    assert (dw == 0).all()


@pytest.mark.parametrize("rows,D,io", [(5000, 64, "bf16"), (3000, 768, "f32"), (300, 20000, "bf16")])
def test_same_bits_every_time(dev, rows, D, io):
    import torch
    X, w, res, dY = make(dev, rows, D, io, 17)
    dX, dw = ttt.rmsnorm_bwd(X, w, dY, res, EPS)
    ws = torch.empty(ttt.rmsnorm_bwd_workspace_bytes(rows, D, int(io == "bf16")), dtype=torch.uint8,
                     device=dev)
    for k in range(5):
        ws.fill_(51 * k)
        a, b = ttt.rmsnorm_bwd(X, w, dY, res, EPS, workspace=ws)
        assert torch.equal(a, dX) and torch.equal(b, dw)


def test_offsets_past_32_bits(dev):
    import torch
    D = 4096
    rows = (1 << 31) // D + 5
    X = torch.zeros(rows, D, dtype=torch.bfloat16, device=dev)
    small, w, _, dY = make(dev, 4, D, "bf16", 19)
    X[-4:] = small
    Y, _ = ttt.rmsnorm_fwd(X, w, None, EPS)
    check_fwd(X[-4:], w, None, Y[-4:], None, "bf16")
    assert (Y[:-4] == 0).all()
    del Y
    Y8, scale, _ = ttt.rmsnorm_q8_fwd(X, w, None, EPS)
    check_q8(X[-4:], w, None, Y8[-4:], scale[-4:], None, "bf16")
    del Y8
    G = torch.zeros_like(X)
    G[-4:] = dY
    dX, dw = ttt.rmsnorm_bwd(X, w, G, None, EPS)
    check_bwd(X[-4:], w, dY, None, dX[-4:], dw, "bf16")
