"""The plain forms of the gated delta rule, group norm and dropout against what they are by other
means: the TTT-Linear oracle at one token a chunk, differences, published test vectors."""
import numpy as np
import pytest

import delta_ref as ref
import oracle


def make(N, T, dk, dv, seed):
    r = np.random.default_rng(seed)
    K, Q = r.standard_normal((N, T, dk)), r.standard_normal((N, T, dk))
    K /= np.linalg.norm(K, axis=2, keepdims=True)
    Q /= np.linalg.norm(Q, axis=2, keepdims=True)
    return (K, Q, r.standard_normal((N, T, dv)), 1 / (1 + np.exp(-r.standard_normal((N, T)))),
            -0.2 * r.random((N, T)), 0.3 * r.standard_normal((N, dv, dk)))


def test_delta_is_ttt_linear_with_one_token_a_chunk():
    K, Q, V, eta, g, W0 = (x.astype(np.float32) for x in make(3, 20, 16, 16, 1))
    Z, W = ref.delta(K, Q, V, eta, 0 * g, W0)[:2]
    Zo, Wo = oracle.linear(K, Q, V, eta, 0.0, W0, 1)
    # the same operations in fp64: 20 tokens of products over 16 features
    assert np.abs(Z - np.asarray(Zo).reshape(Z.shape)).max() <= 1e-12
    assert np.abs(W - np.asarray(Wo).reshape(W.shape)).max() <= 1e-12


def test_delta_starts_anew_where_it_forgets():
    K, Q, V, eta, g, W0 = make(2, 12, 5, 3, 2)
    g[:, 7] = -np.inf
    Z, W = ref.delta(K, Q, V, eta, g, W0)[:2]
    g[:, 7] = 0
    Z2, W2 = ref.delta(K[:, 7:], Q[:, 7:], V[:, 7:], eta[:, 7:], g[:, 7:], 0 * W0)[:2]
    assert np.array_equal(Z[:, 7:], Z2) and np.array_equal(W, W2)


def test_delta_gradients_are_differences():
    args = list(make(1, 9, 4, 3, 3))
    r = np.random.default_rng(4)
    dZ, dW = r.standard_normal(args[2].shape), r.standard_normal(args[5].shape)
    grads = ref.delta_bwd(*args, dZ, dW)
    order = (0, 1, 2, 3, 4, 5)
    loss = lambda a: (ref.delta(*a)[0] * dZ).sum() + (ref.delta(*a)[1] * dW).sum()  # noqa: E731
    for i in order:
        for _ in range(6):
            at = tuple(r.integers(0, n) for n in args[i].shape)
            h, sides = 1e-6, []
            for s in (h, -h):
                a = [x.copy() for x in args]
                a[i][at] += s
                sides.append(loss(a))
            # central differences: h^2 of the third derivative, and 1e-16 / h of the loss
            assert abs((sides[0] - sides[1]) / (2 * h) - grads[i][at]) <= 1e-7


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_groupnorm_gradients_are_differences(act):
    r = np.random.default_rng(5)
    X, dY = r.standard_normal((2, 3, 8)) + 0.5, r.standard_normal((2, 3, 8))
    w, b = 1 + 0.3 * r.standard_normal(8), 0.3 * r.standard_normal(8)
    f = lambda X, w, b: (ref.groupnorm(X, 2, w, b, 1e-5, act)[0] * dY).sum()  # noqa: E731
    _, mean, rstd = ref.groupnorm(X, 2, w, b, 1e-5, act)[:3]
    grads = ref.groupnorm_bwd(X, 2, w, b, dY, mean, rstd, act)[0]
    for i, x in enumerate((X, w, b)):
        for _ in range(6):
            at = tuple(r.integers(0, n) for n in x.shape)
            h, sides = 1e-6, []
            for s in (h, -h):
                a = [X.copy(), w.copy(), b.copy()]
                a[i][at] += s
                sides.append(f(*a))
            assert abs((sides[0] - sides[1]) / (2 * h) - grads[i][at]) <= 1e-7


def test_philox_has_its_published_numbers():
    # the known answers that its authors published with it
    zero, ones = np.zeros((1, 4), np.uint64), np.full((1, 4), 0xFFFFFFFF, np.uint64)
    assert ref.philox(zero, (0, 0)).tolist() == [[0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]]
    assert ref.philox(ones, (0xFFFFFFFF, 0xFFFFFFFF)).tolist() == [
        [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]]
    pi = np.array([[0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]], np.uint64)
    assert ref.philox(pi, (0xA4093822, 0x299F31D0)).tolist() == [
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]]


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9])
def test_dropout_keeps_its_share(p):
    n = 100000
    kept = ref.keep_mask(n, p, 1234, 5).mean()
    # 6 standard deviations of a share of n
    assert abs(kept - (1 - p)) <= 6 * np.sqrt(p * (1 - p) / n)
