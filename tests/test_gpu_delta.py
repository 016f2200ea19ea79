"""GPU parity of the gated delta rule (forward, step, backward) with its token-by-token fp64 form,
within the bounds that delta_ref derives."""
import numpy as np
import pytest

import delta_ref as ref
from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


class Case:
    """Inputs on the GPU in a layout, and in fp64 as [B H, T, d] with a head of keys for each of values."""

    def __init__(self, dev, B, H, share, T, dk, dv, io, layout=ttt.LAYOUT_BHTD, seed=0, forget=(), pad=0,
                 start=True, scale=1.0):
        import torch
        gen = torch.Generator(device="cpu").manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        dt = torch.bfloat16 if io == "bf16" else torch.float32
        self.B, self.H, self.share, self.T, self.dk, self.dv = B, H, share, T, dk, dv
        self.io, self.layout = io, layout
        K, Q = n(B, H // share, T, dk), n(B, H // share, T, dk)
        # (0.99: still at most of unit length after a rounding to bf16)
        K, Q = 0.99 * K / K.norm(dim=3, keepdim=True), 0.99 * Q / Q.norm(dim=3, keepdim=True)
        V, dZ = scale * n(B, H, T, dv), n(B, H, T, dv)
        eta, g = torch.sigmoid(n(B, H, T)), torch.nn.functional.logsigmoid(n(B, H, T) + 3)
        for t in forget:
            g[:, :, t] = -float("inf")
        if pad:
            g[-1:, :, T - pad:] = 0
            eta[-1:, :, T - pad:] = 0
        self.W0 = (0.3 * n(B, H, dv, dk)).to(dev) if start else None
        self.dW = n(B, H, dv, dk).to(dev) if start else None
        lay = (lambda t: t.transpose(1, 2).contiguous()) if layout == ttt.LAYOUT_BTHD else (lambda t: t)
        self.K, self.Q, self.V, self.dZ = (lay(t.to(dt)).to(dev) for t in (K, Q, V, dZ))
        self.eta, self.g = lay(eta).to(dev), lay(g).to(dev)

    def flat(self, t):
        """[B H, T, ...] in fp64 of a token tensor."""
        x = t.double().cpu().numpy()
        x = np.swapaxes(x, 1, 2) if self.layout == ttt.LAYOUT_BTHD else x
        if x.shape[1] != self.H:
            x = np.repeat(x, self.share, 1)
        return np.ascontiguousarray(x.reshape((self.B * self.H,) + x.shape[2:]))

    def state(self, t):
        if t is None:
            return np.zeros((self.B * self.H, self.dv, self.dk))
        return t.double().cpu().numpy().reshape(self.B * self.H, self.dv, self.dk)

    def inputs(self):
        g = self.flat(self.g) if self.g is not None else np.zeros((self.B * self.H, self.T))
        return [self.flat(t) for t in (self.K, self.Q, self.V, self.eta)] + [g, self.state(self.W0)]


def near(name, got, want, io, rel, scale=None):
    """|got - want| <= rel * (largest of the head) + half a step of the type."""
    axes = tuple(range(1, want.ndim))
    big = np.abs(want).max(axes, keepdims=True) if scale is None else scale
    ok, worst = ref.within(got, want, np.broadcast_to(rel * big, want.shape), io)
    say("  %s: error over what is allowed %.3f" % (name, worst))
    assert ok, name


def largest(c, Z, before):
    """What a bf16 Z's left-out products are relative to: the largest read of a head."""
    return np.maximum(np.abs(Z).max((1, 2)), np.abs(before).max((0, 2, 3)))[:, None, None]


def check_fwd(c, Z, W):
    want, last, before, _ = ref.delta(*c.inputs())
    rel = ref.delta_rel(c.T, c.dk, c.dv)
    big = largest(c, want, before)
    near("Z", c.flat(Z), want, c.io, rel + (ref.Z_BF16 if c.io == "bf16" else 0.0), big)
    near("W", c.state(W), last, "f32", rel, big)


FWD = [
    # B, H, share, T, dk, dv
    (1, 1, 1, 1, 64, 64), (1, 1, 1, 2, 16, 16), (2, 2, 1, 16, 64, 64), (2, 3, 1, 17, 64, 64), (1, 2, 1, 63, 32, 48),
    (1, 2, 1, 64, 64, 64), (1, 2, 1, 65, 64, 64), (2, 2, 2, 130, 128, 128), (1, 4, 2, 200, 50, 83),
    (1, 1, 1, 129, 1, 1), (1, 2, 1, 100, 7, 9), (1, 1, 1, 70, 96, 200), (2, 1, 1, 70, 128, 256), (1, 4, 4, 90, 33, 17),
    (3, 5, 1, 300, 64, 32),
]


@pytest.mark.parametrize("layout", [ttt.LAYOUT_BHTD, ttt.LAYOUT_BTHD])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", FWD)
def test_forward(dev, shape, io, layout):
    c = Case(dev, *shape, io, layout, seed=sum(shape))
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, layout=layout))


# few heads and many tokens: sequences in segments
LONG = [(1, 1, 1, 2000, 64, 64), (1, 2, 2, 2600, 128, 128), (2, 1, 1, 1601, 32, 83), (1, 1, 1, 3000, 50, 200)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", LONG)
def test_long_sequences_of_few_heads(dev, shape, io):
    c = Case(dev, *shape, io, ttt.LAYOUT_BTHD, seed=sum(shape), forget=(700, 1500))
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, layout=c.layout))
    check_bwd(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW, layout=c.layout))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("forget", [(0,), (63,), (64,), (10, 11, 64, 65, 140), tuple(range(0, 150, 3)), (149,)])
def test_forward_forgets(dev, io, forget):
    c = Case(dev, 1, 2, 1, 150, 64, 64, io, seed=11, forget=forget)
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0))
    lowest = c.g.masked_fill(c.g == -float("inf"), -3.4028234663852886e38)
    a, b = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0), ttt.delta_fwd(c.K, c.Q, c.V, c.eta, lowest, c.W0)
    assert all((x == y).all() for x, y in zip(a, b))


@pytest.mark.parametrize("T", [9, 200])
def test_forward_without_state_decay_or_sizes(dev, T):
    c = Case(dev, 2, 2, 1, T, 64, 64, "bf16", seed=3, start=False)
    c.g = None
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, c.eta))
    import torch
    c.eta = torch.full_like(c.eta, 0.25)
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, None, eta_scalar=0.25))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_forward_padding_keeps_the_state(dev, io):
    T, pad = 170, 50
    c = Case(dev, 1, 3, 1, T, 64, 64, io, seed=5, pad=pad)
    W = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0)[1]
    s = slice(0, T - pad)
    short = [t[:, :, s].contiguous() for t in (c.K, c.Q, c.V, c.eta, c.g)]
    W2 = ttt.delta_fwd(*short, c.W0)[1]
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0))
    # the same state by chunks that end elsewhere
    big = W.abs().max().item()
    assert (W - W2).abs().max().item() <= 2 * ref.delta_rel(T, 64, 64) * big


@pytest.mark.parametrize("drop", [-2.0, -30.0, -90.0, -200.0, -1e4, -1e12, -9e29])
def test_forward_strong_decays_among_weak_ones(dev, drop):
    """Sums of log decays that are far from 0 before tokens that hardly decay."""
    c = Case(dev, 1, 2, 1, 130, 64, 64, "f32", seed=6)
    c.g[:, :, 5:60:6] = drop
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0))


def test_forward_in_place_state_and_same_bits(dev):
    c = Case(dev, 2, 3, 1, 200, 64, 64, "bf16", seed=8)
    Z, W = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0)
    W1 = c.W0.clone()
    Z1, W2 = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, W1, W_out=W1)
    assert (Z == Z1).all() and (W == W2).all() and W2 is W1


@pytest.mark.parametrize("layout", [ttt.LAYOUT_BHTD, ttt.LAYOUT_BTHD])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 3, 1, 64, 64), (1, 4, 2, 128, 128), (1, 2, 1, 50, 83), (2, 1, 1, 3, 256),
                                   (1, 2, 1, 100, 5), (100, 8, 4, 64, 83), (60, 10, 1, 18, 130), (40, 8, 2, 128, 256)])
def test_step_continues(dev, shape, io, layout):
    B, H, share, dk, dv = shape
    T = 7
    c = Case(dev, B, H, share, T, dk, dv, io, layout, seed=dk, forget=(4,))
    W, axis, Z, at = c.W0.clone(), 2 if layout == ttt.LAYOUT_BHTD else 1, [], 0
    import torch
    for n in (1, 2, 1, 3):
        part = [t.narrow(axis, at, n).clone() for t in (c.K, c.Q, c.V, c.eta, c.g)]
        Z.append(ttt.delta_step(*part, W, layout=layout))
        at += n
    check_fwd(c, torch.cat(Z, axis), W)


BWD = [
    (1, 1, 1, 1, 64, 64), (1, 2, 1, 5, 16, 16), (1, 2, 1, 64, 64, 64), (2, 2, 1, 65, 64, 64), (1, 4, 2, 150, 128, 128),
    (1, 4, 4, 130, 50, 83), (1, 2, 1, 100, 7, 9), (1, 1, 1, 70, 96, 200), (1, 2, 2, 70, 128, 256), (2, 3, 1, 200, 32, 32),
    (1, 1, 1, 66, 1, 1),
]


def check_bwd(c, got):
    args = c.inputs() + [c.flat(c.dZ), c.state(c.dW)]
    want = ref.delta_bwd(*args)
    rel = ref.delta_rel(c.T, c.dk, c.dv)
    keys = [x.reshape(c.B, -1, c.share, c.T, c.dk).sum(2).reshape(-1, c.T, c.dk) for x in want[:2]]
    plain = Case.flat
    share, c.share, H, c.H = c.share, 1, c.H, c.H // c.share
    dK, dQ = plain(c, got[0]), plain(c, got[1])
    c.share, c.H = share, H
    # the gradients' parts are about as large as the largest of them; a head of keys adds up `share`
    near("dK", dK, keys[0], c.io, rel * c.share)
    near("dQ", dQ, keys[1], c.io, rel * c.share)
    near("dV", c.flat(got[2]), want[2], c.io, rel)
    near("deta", c.flat(got[3]), want[3], "f32", rel)
    # dg sums, over its chunk, products of q and dQ and of k and dK's two parts, which cancel
    part = np.abs(want[4]).max(1) + 3 * (np.linalg.norm(want[0], axis=2) * np.linalg.norm(args[0], axis=2)
                                         + np.linalg.norm(want[1], axis=2) * np.linalg.norm(args[1], axis=2)).max(1)
    near("dg", c.flat(got[4]), want[4], "f32", rel, part[:, None])
    near("dW0", c.state(got[5]), want[5], "f32", rel)
    forgets = c.flat(c.g) <= -1e30 if c.g is not None else np.zeros(1, bool)
    assert (c.flat(got[4])[forgets] == 0).all() if c.g is not None else True


@pytest.mark.parametrize("layout", [ttt.LAYOUT_BHTD, ttt.LAYOUT_BTHD])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", BWD)
def test_backward(dev, shape, io, layout):
    c = Case(dev, *shape, io, layout, seed=sum(shape) + 1)
    check_bwd(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW, layout=layout))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("forget", [(0,), (63,), (64,), (10, 11, 64, 65, 140), tuple(range(0, 150, 3)), (149,)])
def test_backward_forgets(dev, io, forget):
    c = Case(dev, 1, 2, 1, 150, 64, 64, io, seed=12, forget=forget, pad=20)
    check_bwd(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW))


def test_backward_without_state_decay_or_sizes(dev):
    c = Case(dev, 2, 2, 1, 130, 64, 64, "bf16", seed=4, start=False)
    c.g = None
    check_bwd(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, None, None, c.dZ))
    import torch
    c.eta = torch.full_like(c.eta, 0.25)
    check_bwd(c, ttt.delta_bwd(c.K, c.Q, c.V, None, None, None, c.dZ, eta_scalar=0.25))


def test_backward_of_steps_that_write_nothing(dev):
    """eta = 0: the token writes nothing, and its step size has a gradient all the same."""
    c = Case(dev, 1, 2, 1, 100, 64, 64, "f32", seed=14)
    c.eta[:, :, 20:50] = 0
    check_bwd(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW))


def test_backward_same_bits(dev):
    c = Case(dev, 2, 4, 2, 200, 64, 64, "bf16", seed=9)
    a = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    b = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    assert all((x == y).all() for x, y in zip(a, b))


def test_non_finite_values_stay_in_their_head(dev):
    c = Case(dev, 1, 3, 1, 150, 64, 64, "bf16", seed=10)
    clean = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0)
    grads = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    c.V[0, 1, 70, 3] = float("nan")
    c.K[0, 1, 90, 5] = float("inf")
    for got, want in zip(ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0)
                         + ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW), clean + grads):
        for h in (0, 2):
            assert (got[0, h] == want[0, h]).all()
    assert ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0)[1][0, 1].isnan().any()


def test_outputs_end_where_they_should(dev):
    """Rows behind the outputs keep what they held."""
    import torch
    c = Case(dev, 1, 2, 1, 70, 50, 83, "bf16", seed=15)
    n = c.V.numel()
    room = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device=dev)
    Z = room[:n].view(c.V.shape)
    ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, Z=Z)
    assert (room[n:] == 7).all()
    outs = [torch.full((t.numel() + 512,), 7.0, dtype=t.dtype, device=dev)
            for t in (c.K, c.Q, c.V, c.eta, c.g, c.W0)]
    views = [o[:t.numel()].view(t.shape) for o, t in zip(outs, (c.K, c.Q, c.V, c.eta, c.g, c.W0))]
    ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW,
                  **dict(zip(("dK", "dQ", "dV", "deta", "dg", "dW0"), views)))
    assert all((o[t.numel():] == 7).all() for o, t in zip(outs, views))


@pytest.mark.parametrize("shape", [(1, 1, 1, 4000, 64, 64), (1, 32, 1, 8192, 64, 64), (1, 2, 1, 3000, 128, 128)])
def test_forward_in_place_in_segments(dev, shape):
    """W_out at W0's place where the sequence's segments run at once: the first reads its state from
    elsewhere."""
    c = Case(dev, *shape, "bf16", seed=31)
    Z, W = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0)
    for _ in range(3):
        W1 = c.W0.clone()
        Z1, _ = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, W1, W_out=W1)
        assert (Z == Z1).all() and (W == W1).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(10, 16, 1, 130, 64, 64), (5, 32, 2, 70, 32, 64), (10, 16, 1, 140, 128, 60),
                                   (3, 32, 4, 100, 50, 83)])
def test_many_heads(dev, shape, io):
    """Enough heads for workgroups of 64 columns."""
    c = Case(dev, *shape, io, seed=sum(shape), forget=(66,))
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0))
    check_bwd(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 32, 1, 8192, 64, 64), (1, 32, 1, 8200, 32, 50), (1, 24, 1, 12000, 128, 64),
                                   (1, 24, 1, 8192, 32, 64)])
def test_segments_of_many_heads(dev, shape, io):
    """Sequences in segments with workgroups of 64 columns: as a few heads at a time."""
    B, H, share, T, dk, dv = shape
    c = Case(dev, *shape, io, seed=sum(shape), forget=(1000, 5000))
    whole = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0) + ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    rel = 2 * ref.delta_rel(T, dk, dv)
    # (dg's parts cancel: about ten times its largest value goes into the sum)
    more = {0: ref.HALF[io] * 2 + (2 * ref.Z_BF16 if io == "bf16" else 0), 2: 2 * ref.HALF[io], 3: 2 * ref.HALF[io],
            4: 2 * ref.HALF[io], 6: 9 * rel}
    for h in range(0, H, 4):
        s = slice(h, h + 4)
        part = [t[:, s].contiguous() for t in (c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)]
        alone = ttt.delta_fwd(*part[:6]) + ttt.delta_bwd(*part)
        for i, (a, b) in enumerate(zip(whole, alone)):
            err = (a[:, s].double() - b.double()).abs().max().item()
            assert err <= (rel + more.get(i, 0)) * b.double().abs().max().item(), (h, i, err)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 3, 1, 40, 64, 64), (1, 2, 1, 33, 128, 1), (1, 2, 2, 90, 2, 256)])
def test_step_of_many_tokens(dev, shape, io):
    c = Case(dev, *shape, io, seed=44, forget=(20,))
    W = c.W0.clone()
    Z = ttt.delta_step(c.K, c.Q, c.V, c.eta, c.g, W)
    check_fwd(c, Z, W)


def test_one_tensor_for_keys_queries_and_values(dev):
    c = Case(dev, 1, 2, 1, 100, 64, 64, "f32", ttt.LAYOUT_BTHD, seed=45)
    c.Q = c.V = c.K
    check_fwd(c, *ttt.delta_fwd(c.K, c.K, c.K, c.eta, c.g, c.W0, layout=c.layout))
    check_bwd(c, ttt.delta_bwd(c.K, c.K, c.K, c.eta, c.g, c.W0, c.dZ, c.dW, layout=c.layout))


def test_backward_leaves_out_what_is_not_asked_for(dev):
    """deta, dg and dW0 are optional in the C call; a shared head's sums are not."""
    import torch
    c = Case(dev, 1, 4, 2, 100, 64, 64, "bf16", seed=46)
    want = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    dK, dQ, dV = (torch.empty_like(t) for t in (c.K, c.Q, c.V))
    n = ttt.delta_bwd_workspace_bytes(1, 4, 2, 100, 64, 64, 1)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    p = lambda t: t.data_ptr()  # noqa: E731
    rc = ttt.lib().ttt_delta_bwd(p(c.K), p(c.Q), p(c.V), p(c.eta), 0.0, p(c.g), p(c.W0), p(c.dZ), p(c.dW), p(dK), p(dQ),
                                 p(dV), None, None, None, 1, 4, 2, 100, 64, 64, 0, 1, p(ws), n,
                                 torch.cuda.current_stream().cuda_stream)
    assert rc == ttt.OK
    assert all((a == b).all() for a, b in zip((dK, dQ, dV), want))
