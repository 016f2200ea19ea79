"""The gradient of the gated delta rule's decays where decays are strong: a token's has the digits of
what crosses it, however large the chunk's other products are."""
import numpy as np
import pytest

import delta_ref as ref
from gpu_helpers import say
from test_gpu_delta import Case, LONG, check_bwd
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def crossing(K, Q, V, eta, g, W0, dZ, dW):
    """dg in fp64, and for every token the sum of the absolute products it is made of: the state's
    gradient right after the decay times the decayed state, taken apart into what each later read
    and each earlier write brings."""
    K, Q, V, eta, g, W0, dZ, dW = (np.asarray(x, np.float64) for x in (K, Q, V, eta, g, W0, dZ, dW))
    dK, _, dV, _, dg, _ = ref.delta_bwd(K, Q, V, eta, g, W0, dZ, dW)
    u = ref.delta(K, Q, V, eta, g, W0)[3]
    N, T, _ = K.shape
    size = np.zeros((N, T))
    with np.errstate(divide="ignore"):
        a = np.where(g <= -1e30, 0.0, np.exp(g))
    # writes (eta u_r, k_r) and the first state's rows; reads (dZ_s, q_s), (-dV_s, k_s) and the last one's
    for n in range(N):
        E = np.zeros((T + 2, T + 1))           # decay from after write r (0: the first state) to read s
        for r in range(T + 1):
            E[r, r] = 1.0
            for s in range(r + 1, T + 2):
                E[s, r] = E[s - 1, r] * (a[n, s - 1] if s <= T else 1.0)
        w = eta[n, :, None] * u[n]
        last = np.abs(dW[n])
        M = np.zeros((T + 2, T + 1))
        M[1:T + 1, 1:] = np.abs((dZ[n] @ w.T) * (Q[n] @ K[n].T)) + np.abs((dV[n] @ w.T) * (K[n] @ K[n].T))
        M[T + 1, 1:] = np.abs(np.einsum("tv,vk,tk->t", np.abs(w), last, np.abs(K[n])))
        M[1:T + 1, 0] = np.einsum("tv,vk,tk->t", np.abs(dZ[n]), np.abs(W0[n]), np.abs(Q[n])) + np.einsum(
            "tv,vk,tk->t", np.abs(dV[n]), np.abs(W0[n]), np.abs(K[n]))
        M[T + 1, 0] = (last * np.abs(W0[n])).sum()
        M *= E
        for t in range(1, T + 1):
            size[n, t - 1] = M[t:, :t].sum()
    return dg, size


def check_dg(c, got):
    """|error| <= delta_rel of the largest such sum of the head.  (A decay over x has the rounding of
    x log2(e), at most 24 U for |x| <= 20, next to delta_rel's 200 U and more.)"""
    args = c.inputs() + [c.flat(c.dZ), c.state(c.dW)]
    want, size = crossing(*args)
    big = size.max(1, keepdims=True)
    err = np.abs(c.flat(got) - want)
    say("  dg: error over what is allowed %.3f" % (err / (ref.delta_rel(c.T, c.dk, c.dv) * big)).max())
    assert (err <= ref.delta_rel(c.T, c.dk, c.dv) * big).all()
    # and nothing where nothing crosses
    assert (c.flat(got)[size == 0] == 0).all()
    return size


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2, 1, 64, 64, 64), (1, 2, 2, 100, 32, 48), (1, 2, 1, 70, 128, 128)])
@pytest.mark.parametrize("g", [-5.0, -10.0, -20.0])
def test_every_decay_is_strong(dev, g, shape, io):
    c = Case(dev, *shape, io, seed=61)
    c.g += g
    check_dg(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)[4])


@pytest.mark.parametrize("start", [True, False])
@pytest.mark.parametrize("g", [-2.0, -15.0])
def test_strong_decays_without_states(dev, g, start):
    """No state crosses the chunk's ends: pairs of its tokens alone."""
    c = Case(dev, 1, 3, 1, 64, 64, 64, "f32", seed=62, start=start)
    c.g += g
    if start:
        c.W0, c.dW = 0 * c.W0, 0 * c.dW
    check_dg(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)[4])


@pytest.mark.parametrize("drop", [-2.0, -30.0, -90.0, -200.0, -1e4, -1e12, -9e29])
def test_strong_decays_among_weak_ones(dev, drop):
    c = Case(dev, 1, 2, 1, 130, 64, 64, "f32", seed=6)
    c.g[:, :, 5:60:6] = drop
    got = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    check_bwd(c, got)
    size = check_dg(c, got[4])
    # no more than the absolute products come to (twice: their factors have roundings of their own;
    # 1e-35: a decay below fp32's normal numbers may keep its last digits or not)
    assert (np.abs(c.flat(got[4])) <= 2 * size + 1e-35).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [60, 150])
def test_documents_without_a_gradient(dev, T, io):
    """A document that no gradient reaches, between ones that it reaches: its gradients are 0."""
    at = (10, 25, 40)
    c = Case(dev, 1, 2, 1, T, 64, 64, io, seed=63, forget=at)
    c.dZ[:, :, at[0]:at[1]] = 0
    c.dZ[:, :, at[1]:at[2]] = 0
    got = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    check_dg(c, got[4])
    for name, x in zip(("dK", "dQ", "dV", "deta", "dg"), got):
        assert (x[:, :, at[0]:at[2]] == 0).all(), name


@pytest.mark.parametrize("shape", [(2, 3, 1, 1, 64, 64), (1, 2, 1, 17, 33, 17), (1, 4, 4, 130, 50, 83),
                                   (1, 1, 1, 129, 1, 1), (12, 16, 1, 66, 64, 64), (1, 2, 1, 70, 128, 256)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_weak_decays(dev, shape, io):
    c = Case(dev, *shape, io, ttt.LAYOUT_BTHD, seed=sum(shape))
    if shape[0] * shape[1] > 8:
        c.g[:, 0::2] -= 8
    check_dg(c, ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW, layout=c.layout)[4])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_decays_in_segments(dev, io):
    """Sequences in segments, every eighth token a strong decay: against the tokens' own fp64 form."""
    shape = LONG[0]
    c = Case(dev, *shape, io, ttt.LAYOUT_BTHD, seed=64)
    c.g[:, ::8] -= 12
    got = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW, layout=c.layout)
    want = ref.delta_bwd(*c.inputs(), c.flat(c.dZ), c.state(c.dW))[4]
    # products that cross a token add up to some ten times the largest gradient here
    assert (np.abs(c.flat(got[4]) - want).max(1) <= 10 * ref.delta_rel(c.T, c.dk, c.dv) * np.abs(want).max(1)).all()
