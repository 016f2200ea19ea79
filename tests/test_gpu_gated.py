"""GPU parity of the gated linear recurrence (forward, step, backward) with its fp64 form, within
the bounds that block_ref derives."""
import numpy as np
import pytest

import block_ref as ref
from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def dtype(io):
    import torch
    return torch.bfloat16 if io == "bf16" else torch.float32


def make(dev, N, T, d, io, seed, resets=0, pad=0, start=True, bias=3.0):
    """X, G [1, N, T, d] and h0 [1, N, d] (or None) on the device, as a trained layer has them."""
    import torch
    gen = torch.Generator(device="cpu").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    G = torch.nn.functional.logsigmoid(rnd(1, N, T, d) + bias)
    X = rnd(1, N, T, d)
    for k in range(resets):
        G[:, :, (k * 37 + 5 * k * k) % T] = -float("inf")
    if pad:
        G[:, -1, T - pad:] = 0
        X[:, -1, T - pad:] = 0
    h0 = rnd(1, N, d).to(dev) if start else None
    return X.to(dev, dtype(io)), G.to(dev, dtype(io)), h0


def np64(t):
    return t.double().cpu().numpy()[0]


def state(h, like):
    return np.zeros((like.shape[1], like.shape[3])) if h is None else np64(h)


def check_fwd(X, G, h0, Z, hT, io):
    x, g, h = np64(X), np64(G), state(h0, X)
    want, bound = ref.gated(x, g, h), ref.gated_bound(x, g, h)
    ok, worst = ref.within(np64(Z), want, bound, io)
    ok2, worst2 = ref.within(np64(hT), want[:, -1], bound[:, -1], "f32")
    say("  error over what is allowed: Z %.3f h_T %.3f" % (worst, worst2))
    assert ok and ok2


def check_bwd(dev, G, Z, h0, io, seed, dhT=True):
    import torch
    gen = torch.Generator(device="cpu").manual_seed(seed)
    dZ = torch.randn(G.shape, generator=gen).to(dev, G.dtype)
    dh = torch.randn(G.shape[0], G.shape[1], G.shape[3], generator=gen).to(dev) if dhT else None
    got = ttt.gated_bwd(G, Z, dZ, h0, dh)
    torch.cuda.synchronize()
    args = (np64(G), np64(Z), state(h0, G), np64(dZ), state(dh, G))
    want, bound = ref.gated_bwd(*args), ref.gated_bwd_bound(*args)
    for k, name in enumerate(("dX", "dG", "dh0")):
        ok, worst = ref.within(np64(got[k]), want[k], bound[k], "f32" if k == 2 else io)
        say("  error over what is allowed: %s %.3f" % (name, worst))
        assert ok, name
    return got


LENGTHS = [1, 2, 7, 8, 9, 31, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1000, 2049]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(dev, T, io):
    say("case T", T, io)
    X, G, h0 = make(dev, 5, T, 64, io, 100 + T)
    Z, hT = ttt.gated_fwd(X, G, h0)
    check_fwd(X, G, h0, Z, hT, io)
    check_bwd(dev, G, Z, h0, io, 200 + T)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 2, 3, 4, 8, 12, 16, 24, 32, 33, 50, 72, 83, 100, 128, 200, 257, 520])
def test_widths(dev, d, io):
    say("case d", d, io)
    for T, N in ((1, 3), (300, 3), (700, 2)):
        X, G, h0 = make(dev, N, T, d, io, 300 + d, resets=2, pad=T // 7)
        Z, hT = ttt.gated_fwd(X, G, h0)
        check_fwd(X, G, h0, Z, hT, io)
        check_bwd(dev, G, Z, h0, io, 400 + d)


@pytest.mark.parametrize("N,T,d,io", [(96, 520, 64, "bf16"), (2, 20011, 64, "bf16"), (1, 9000, 3, "f32"),
                                      (300, 70, 16, "bf16"), (300, 400, 64, "bf16"), (40, 500, 128, "f32"), (1, 40000, 1, "bf16"), (7, 3001, 83, "f32")])
def test_sizes(dev, N, T, d, io):
    say("case", N, T, d, io)
    X, G, h0 = make(dev, N, T, d, io, 500, resets=3)
    Z, hT = ttt.gated_fwd(X, G, h0)
    check_fwd(X, G, h0, Z, hT, io)
    check_bwd(dev, G, Z, h0, io, 501)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_no_states_given(dev, io):
    import torch
    X, G, _ = make(dev, 4, 600, 64, io, 7, start=False)
    Z, hT = ttt.gated_fwd(X, G)
    check_fwd(X, G, None, Z, hT, io)
    got = check_bwd(dev, G, Z, None, io, 8, dhT=False)
    # the C entry takes NULL for h_out and dh0 too, and then writes neither
    Z2, dX, dG = torch.empty_like(Z), torch.empty_like(Z), torch.empty_like(Z)
    ws = torch.empty(max(1, ttt.gated_workspace_bytes(1, 4, 600, 64, int(io == "bf16"))),
                     dtype=torch.uint8, device=dev)
    st = torch.cuda.current_stream().cuda_stream
    L = ttt.lib()
    assert L.ttt_gated_fwd(X.data_ptr(), G.data_ptr(), None, Z2.data_ptr(), None, 1, 4, 600, 64,
                           int(io == "bf16"), ws.data_ptr(), ws.numel(), st) == ttt.OK
    gen = torch.Generator(device="cpu").manual_seed(8)
    dZ = torch.randn(G.shape, generator=gen).to(dev, G.dtype)
    assert L.ttt_gated_bwd(G.data_ptr(), Z.data_ptr(), None, dZ.data_ptr(), None, dX.data_ptr(),
                           dG.data_ptr(), None, 1, 4, 600, 64, int(io == "bf16"), ws.data_ptr(),
                           ws.numel(), st) == ttt.OK
    assert torch.equal(Z, Z2) and torch.equal(dX, got[0]) and torch.equal(dG, got[1])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gates_at_their_ends(dev, io):
    """Gates of 1 over a whole sequence (the state is a running sum), gates that underflow, and all
    shut."""
    X, G, h0 = make(dev, 3, 1500, 64, io, 21)
    for value in (0.0, -200.0, -float("inf"), -1e-4):
        G.fill_(value)
        say("case g =", value)
        Z, hT = ttt.gated_fwd(X, G, h0)
        check_fwd(X, G, h0, Z, hT, io)
        check_bwd(dev, G, Z, h0, io, 22)


@pytest.mark.parametrize("at", [0, 1, 8, 255, 256, 300, 1023, 1024, 1099])
def test_what_is_not_finite_ends_at_a_reset(dev, at):
    """NaN, infinities and a NaN gate pass through the states up to the next reset and no further, in
    their own channels alone."""
    import torch
    X, G, h0 = make(dev, 2, 1100, 64, "f32", 31, resets=0)
    first = max(0, at - 40)
    X[0, 0, first, 3] = float("nan")
    X[0, 0, first, 4] = float("inf")
    G[0, 1, first, 5] = float("nan")
    h0[0, 1, 6] = float("nan")
    G[:, :, at] = -float("inf")
    if first == at:          # the reset's own x: what it holds stays in
        say("reset on the value itself")
    Z, hT = ttt.gated_fwd(X, G, h0)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        want = ref.gated(np64(X), np64(G), np64(h0))
    z = np64(Z)
    assert np.array_equal(np.isnan(z), np.isnan(want))
    clean = [c for c in range(64) if c not in (3, 4, 5, 6)]
    x, g, h = np64(X)[..., clean], np64(G)[..., clean], np64(h0)[..., clean]
    assert ref.within(z[..., clean], want[..., clean], ref.gated_bound(x, g, h), "f32")[0]
    inf = np.isposinf(want[0, :, 4])
    assert np.array_equal(np.isfinite(z[0, :, 4]), ~inf)
    # and backward: a shut gate hands nothing back
    dZ = torch.ones_like(X)
    dZ[0, 0, min(1099, at + 3), 9] = float("nan")
    Zf = torch.nan_to_num(Z, 0.0, 0.0, 0.0)
    got = ttt.gated_bwd(G.nan_to_num(0.0, 0.0, -float("inf")), Zf, dZ, None, None)
    torch.cuda.synchronize()
    gg = np.where(np.isnan(np64(G)), 0.0, np64(G))
    wx, wg, wh = ref.gated_bwd(gg, np64(Zf), np.zeros((2, 64)), np64(dZ), np.zeros((2, 64)))
    for got_k, want_k in zip(got, (wx, wg, wh)):
        assert np.array_equal(np.isnan(np64(got_k)), np.isnan(want_k))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [12, 700])
def test_the_lowest_value_is_a_reset(dev, T, io):
    """Masks of a type's lowest value, and of -1e30, forget like -inf, bit for bit and NaN included."""
    import torch
    X, G, h0 = make(dev, 3, T, 64, io, 33)
    X[0, 0, 2, 5] = float("nan")
    h0[0, 1, 7] = float("inf")
    want = None
    for value in (-float("inf"), torch.finfo(G.dtype).min, -1.01e30):
        G[:, :, 5] = value
        G[:, :, T - 3] = value
        G[:, :, T // 2] = value
        Z, hT = ttt.gated_fwd(X, G, h0)
        back = ttt.gated_bwd(G, Z.nan_to_num(0.0, 0.0, 0.0), X.nan_to_num(0.0, 0.0, 0.0), None, None)
        got = [t.nan_to_num(3.0, 4.0, 5.0) for t in (Z, hT) + back]
        assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
        assert torch.isfinite(Z[:, :, 5:]).all()
        assert all((back[1][:, :, t] == 0).all() for t in (5, T // 2, T - 3))


def test_packed_documents_are_the_separate_ones(dev):
    import torch
    lens = [1, 255, 256, 7, 600, 1, 1, 300]
    X, G, _ = make(dev, 2, sum(lens), 64, "f32", 41)
    t = 0
    for n in lens:
        G[:, :, t] = -float("inf")
        t += n
    Z, _ = ttt.gated_fwd(X, G)
    t = 0
    for n in lens:
        z, _ = ttt.gated_fwd(X[:, :, t:t + n].contiguous(), G[:, :, t:t + n].contiguous())
        torch.cuda.synchronize()
        x, g = np64(X)[:, t:t + n], np64(G)[:, t:t + n]
        assert ref.within(np64(Z)[:, t:t + n], np64(z), 2 * ref.gated_bound(x, g, np.zeros((2, 64))),
                          "f32")[0]
        t += n


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 50])
def test_step_continues_the_sequence(dev, io, d):
    import torch
    X, G, h0 = make(dev, 6, 40, d, io, 51, resets=2)
    h = h0.clone()
    Zs, t = [], 0
    for n in (1, 1, 3, 1, 9, 25):
        Zs.append(ttt.gated_step(X[:, :, t:t + n].contiguous(), G[:, :, t:t + n].contiguous(), h))
        t += n
    torch.cuda.synchronize()
    check_fwd(X, G, h0, torch.cat(Zs, 2), h, io)


@pytest.mark.parametrize("N,T,d,io", [(5000, 40, 64, "bf16"), (700, 60, 200, "f32"), (3000, 17, 50, "bf16")])
def test_many_short_rows(dev, N, T, d, io):
    """Rows that the serial kernel takes, and some that it does not."""
    say("case", N, T, d, io)
    X, G, h0 = make(dev, N, T, d, io, 55, resets=1)
    Z, hT = ttt.gated_fwd(X, G, h0)
    check_fwd(X, G, h0, Z, hT, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [3, 9, 83, 261, 520, 1029])
@pytest.mark.parametrize("T", [1, 5, 40, 900])
def test_state_in_place_at_any_width(dev, T, d, io):
    """h_out at h0's place where the threads' channels do not divide the row: no channel's state is
    read after it is written."""
    import torch
    X, G, h0 = make(dev, 6, T, d, io, 57)
    Z, hT = ttt.gated_fwd(X, G, h0)
    for k in range(3):
        h = h0.clone()
        Z2, _ = ttt.gated_fwd(X, G, h, h_out=h)
        torch.cuda.synchronize()
        assert torch.equal(Z, Z2) and torch.equal(hT, h)
    check_fwd(X, G, h0, Z, hT, io)
    h = h0.clone()
    Z3 = ttt.gated_step(X, G, h)
    torch.cuda.synchronize()
    check_fwd(X, G, h0, Z3, h, io)


def test_state_in_place(dev):
    """h_out at h0's place, over several tiles of a sequence."""
    import torch
    X, G, h0 = make(dev, 40, 2500, 64, "bf16", 61)
    Z, hT = ttt.gated_fwd(X, G, h0)
    h = h0.clone()
    Z2, h2 = ttt.gated_fwd(X, G, h, h_out=h)
    torch.cuda.synchronize()
    assert h2 is h and torch.equal(Z, Z2) and torch.equal(hT, h)


@pytest.mark.parametrize("N,T,d,io", [(32, 9000, 64, "bf16"), (3, 5000, 83, "f32"), (1, 30000, 16, "f32")])
def test_same_bits_every_time(dev, N, T, d, io):
    import torch
    X, G, h0 = make(dev, N, T, d, io, 71)
    dZ = X.flip(2).contiguous()
    Z, hT = ttt.gated_fwd(X, G, h0)
    grads = ttt.gated_bwd(G, Z, dZ, h0, hT)
    ws = torch.empty(max(1, ttt.gated_workspace_bytes(1, N, T, d, int(io == "bf16"))),
                     dtype=torch.uint8, device=dev)
    for k in range(6):
        ws.fill_(37 * k)                # what an earlier call left there does not matter
        Z2, h2 = ttt.gated_fwd(X, G, h0, workspace=ws)
        assert torch.equal(Z, Z2) and torch.equal(hT, h2)
        for a, b in zip(grads, ttt.gated_bwd(G, Z, dZ, h0, hT, workspace=ws)):
            assert torch.equal(a, b)


def test_writes_its_outputs_alone(dev):
    """Outputs inside larger buffers: what is around them stays."""
    import torch
    N, T, d = 3, 333, 72
    X, G, h0 = make(dev, N, T, d, "bf16", 81)
    n = X.numel()
    for size in (n,):
        buf = torch.full((n + 4096,), 7.0, dtype=torch.bfloat16, device=dev)
        Z = buf[2048:2048 + n].view(X.shape)
        hb = torch.full((N * d + 512,), 7.0, device=dev)
        hT = hb[256:256 + N * d].view(1, N, d)
        ttt.gated_fwd(X, G, h0, Z=Z, h_out=hT)
        torch.cuda.synchronize()
        assert (buf[:2048] == 7).all() and (buf[2048 + n:] == 7).all()
        assert (hb[:256] == 7).all() and (hb[256 + N * d:] == 7).all()
        check_fwd(X, G, h0, Z, hT, "bf16")


def test_gradient_is_the_difference_quotient(dev):
    """The kernels' own forward pass, fp32, moved along a direction: the difference of <dZ, Z> is the
    gradient's product with it.  Linear in X and h0, so the step may be large there: what remains are
    roundings, at most the forward bound at both ends."""
    import torch
    X, G, h0 = make(dev, 4, 700, 64, "f32", 91)
    Z, hT = ttt.gated_fwd(X, G, h0)
    gen = torch.Generator(device="cpu").manual_seed(92)
    dZ = torch.randn(X.shape, generator=gen).to(dev)
    dX, dG, dh0 = ttt.gated_bwd(G, Z, dZ, h0, None)
    V = torch.randn(X.shape, generator=gen).to(dev)
    Z2, _ = ttt.gated_fwd(X + V, G, h0)
    diff = (dZ.double() * (Z2.double() - Z.double())).sum().item()
    along = (dX.double() * ((X + V).double() - X.double())).sum().item()
    bound = sum(ref.gated_bound(np64(x), np64(G), np64(h0)) for x in (X, X + V))
    bound = bound + ref.HALF["f32"] * (np.abs(np64(Z)) + np.abs(np64(Z2)))
    e = ref.gated_bwd_bound(np64(G), np64(Z), np64(h0), np64(dZ), np.zeros((4, 64)))[0]
    room = (np.abs(np64(dZ)) * bound).sum() + ((e + ref.HALF["f32"] * np.abs(np64(dX))) * np.abs(np64(V))).sum()
    say("difference %.6g gradient %.6g allowed %.3g" % (diff, along, room))
    assert abs(diff - along) <= room


def test_offsets_past_32_bits(dev):
    """More than 2^31 elements in one row: the last tokens, after a reset, are right."""
    import torch
    d, T, tail = 128, (1 << 24) + 4099, 60
    X = torch.zeros(1, 1, T, d, dtype=torch.bfloat16, device=dev)
    G = torch.full((1, 1, T, d), -0.25, dtype=torch.bfloat16, device=dev)
    gen = torch.Generator(device="cpu").manual_seed(93)
    X[:, :, -tail:] = torch.randn(1, 1, tail, d, generator=gen).to(dev)
    X[:, :, 0] = 1.0
    G[:, :, -tail] = -float("inf")
    say("elements", X.numel())
    Z, hT = ttt.gated_fwd(X, G)
    torch.cuda.synchronize()
    x, g = np64(X[:, :, -tail:]), np64(G[:, :, -tail:])
    want, bound = ref.gated(x, g, np.zeros((1, d))), ref.gated_bound(x, g, np.zeros((1, d)))
    assert ref.within(np64(Z[:, :, -tail:]), want, bound, "bf16")[0]
    assert ref.within(np64(hT), want[:, -1], bound[:, -1], "f32")[0]
    assert np.allclose(np64(Z[:, :, :4])[0, :, 0], np.exp([0.0, -0.25, -0.5, -0.75]), rtol=2.0 ** -7)
    dZ = torch.zeros_like(X)
    dZ[:, :, -1] = 1.0
    dX, dG, dh0 = ttt.gated_bwd(G, Z, dZ)
    torch.cuda.synchronize()
    zr, dz = np64(Z[:, :, -tail:]), np64(dZ[:, :, -tail:])
    args = (g, zr, np.zeros((1, d)), dz, np.zeros((1, d)))
    wx, wg, _ = ref.gated_bwd(*args)
    bx, bg, _ = ref.gated_bwd_bound(*args)
    assert ref.within(np64(dX[:, :, -tail:]), wx, bx, "bf16")[0]
    assert ref.within(np64(dG[:, :, -tail:]), wg, bg, "bf16")[0]
    assert (dX[:, :, :-tail] == 0).all() and (dh0 == 0).all()


@pytest.mark.parametrize("op,BH,T,d", [("fwd", (1 << 22) + 3, 2049, 1), ("fwd", (1 << 23) + 5, 65, 1),
                                       ("step", (1 << 30) + 5, 1, 3), ("bwd", (1 << 23) + 5, 1, 1),
                                       ("bwd", (1 << 22) + 3, 2049, 1)])
def test_more_rows_than_a_grid_holds(dev, op, BH, T, d):
    """Rows that one launch has no room for: those at both ends and on both sides of every place where
    a launch may end have the bits that a call of their own gives them."""
    import torch
    say(op, BH, T, d)
    edge = BH - 20
    picked = torch.tensor([0, 1, *range(edge, BH)], device=dev)
    gen = torch.Generator(device="cpu").manual_seed(BH + T)

    def filled(shape, dtype, of):
        full = torch.full(shape, -0.5, dtype=dtype, device=dev)
        few = of(torch.randn(1, len(picked), *shape[2:], generator=gen)).to(dtype).to(dev)
        full[:, picked] = few
        return full, few

    bf = torch.bfloat16
    X, x = filled((1, BH, T, d), bf, lambda v: v)
    G, g = filled((1, BH, T, d), bf, lambda v: -v.abs())
    h, hs = filled((1, BH, d), torch.float32, lambda v: v)
    if op == "step":
        got, want = [ttt.gated_step(X, G, h), h], [ttt.gated_step(x, g, hs), hs]
    elif op == "fwd":
        got, want = ttt.gated_fwd(X, G, h), ttt.gated_fwd(x, g, hs)
    else:
        got, want = ttt.gated_bwd(G, X, X, h, h), ttt.gated_bwd(g, x, x, hs, hs)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[:, picked], b)
