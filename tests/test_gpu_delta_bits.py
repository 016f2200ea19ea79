"""A bf16 Z of the gated delta rule has the digits of fp32 products behind its own rounding: reads
that nearly cancel, whose last digits are in the operands' last bits."""
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


def state(K, Q, V, eta, W0, r):
    """z = x (a - b), a and b of 24 bits that differ in their last 7."""
    a = (1 + r.random(W0.shape[:3])).astype(np.float32)
    W0[..., 0], W0[..., 1] = a, -(a - np.float32(2.0 ** -23) * r.integers(1, 128, a.shape).astype(np.float32))
    Q[..., 0] = Q[..., 1] = 2.0 ** r.integers(-2, 3, Q.shape[:3])
    return 8.0


def writes(K, Q, V, eta, W0, r):
    """z = x v (eta_0 - eta_1): what two tokens wrote, the step sizes differ in their last 4 bits."""
    K[:, :, 0, 0] = K[:, :, 1, 1] = 1
    V[:, :, 0] = 1 + r.integers(0, 128, V[:, :, 0].shape) / 128
    V[:, :, 1] = -V[:, :, 0]
    eta[:, :, 0] = 0.5 + 0.5 * r.random(eta[:, :, 0].shape)
    eta[:, :, 1] = eta[:, :, 0] - np.float32(2.0 ** -24) * r.integers(1, 16, eta[:, :, 0].shape).astype(np.float32)
    Q[:, :, 2:, 0] = Q[:, :, 2:, 1] = 2.0 ** r.integers(-2, 3, Q[:, :, 2:].shape[:3])
    return 8.0


def pairs(K, Q, V, eta, W0, r):
    """z = v (q.k_0 - q.k_1) / 2, the two products differ in their 17th to 23rd bits: the second
    token's value is 0, so that with step sizes of a half it takes back what the first one wrote."""
    K[:, :, 0, :3] = 1
    K[:, :, 1, :2] = 1
    V[:, :, 0] = 1 + r.integers(0, 128, V[:, :, 0].shape) / 128
    eta[:, :, :2] = 0.5
    Q[:, :, 2:, 0], Q[:, :, 2:, 1] = 1, 1.5 * 2.0 ** -9
    Q[:, :, 2:, 2] = 2.0 ** -23 * r.integers(1, 128, Q[:, :, 2:, 2].shape)
    return 1.0


@pytest.mark.parametrize("shape", [(1, 2, 80, 64, 64), (2, 2, 130, 32, 32), (1, 2, 100, 128, 128), (10, 16, 70, 64, 64),
                                   (10, 16, 70, 128, 64), (1, 1, 2000, 64, 64)])
@pytest.mark.parametrize("case", [state, writes, pairs])
def test_products_behind_a_bf16_output(dev, case, shape):
    import torch
    B, H, T, dk, dv = shape
    K, Q, V = np.zeros((B, H, T, dk)), np.zeros((B, H, T, dk)), np.zeros((B, H, T, dv))
    eta, W0 = np.zeros((B, H, T), np.float32), np.zeros((B, H, dv, dk), np.float32)
    big = case(K, Q, V, eta, W0, np.random.default_rng(sum(shape)))
    t = lambda x, dt: torch.from_numpy(x).to(dt).to(dev)  # noqa: E731
    io = [t(x, torch.bfloat16) for x in (K, Q, V)]
    assert all((x.double().cpu().numpy() == y).all() for x, y in zip(io, (K, Q, V)))    # exact in bf16
    Z, W = ttt.delta_fwd(*io, t(eta, torch.float32), None, t(W0, torch.float32))
    flat = lambda x: x.reshape((B * H,) + x.shape[2:])  # noqa: E731
    want, last = ref.delta(*(flat(x) for x in (K, Q, V, eta)), np.zeros((B * H, T)), flat(W0))[:2]
    # two terms of `big` at most that cancel: a rounding of each on its way (an operand's or the
    # chunk's product, the state's), and of their sums, 8 U of each
    for name, got, ref_, t in (("Z", Z, want, "bf16"), ("W", W, last, "f32")):
        ok, worst = ref.within(flat(got.double().cpu().numpy()), ref_, np.full(ref_.shape, 16 * big * ref.U), t)
        say("  %s: error over what is allowed %.3f" % (name, worst))
        assert ok, name
