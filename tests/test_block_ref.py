"""The fp64 forms that the GPU tests compare with, against central differences."""
import numpy as np
import pytest

import block_ref as ref


def slope(f, x, v, e=1e-6):
    return (f(x + e * v) - f(x - e * v)) / (2 * e)


@pytest.mark.parametrize("T,reset", [(1, False), (5, False), (9, True)])
def test_gated_gradients(T, reset):
    rng = np.random.default_rng(3)
    N, d = 2, 3
    X, G = rng.normal(size=(N, T, d)), -np.abs(rng.normal(size=(N, T, d)))
    if reset:
        G[:, T // 2] = -np.inf
        G[1, 0] = -np.inf
    h0, dZ, dhT = rng.normal(size=(N, d)), rng.normal(size=(N, T, d)), rng.normal(size=(N, d))

    def loss(X, G, h0):
        Z = ref.gated(X, G, h0)
        return (dZ * Z).sum() + (dhT * Z[:, -1]).sum()

    dX, dG, dh0 = ref.gated_bwd(G, ref.gated(X, G, h0), h0, dZ, dhT)
    v = rng.normal(size=X.shape)
    assert np.isclose(slope(lambda x: loss(x, G, h0), X, v), (dX * v).sum(), rtol=1e-7)
    v = np.where(np.isneginf(G), 0.0, rng.normal(size=X.shape))
    assert np.isclose(slope(lambda g: loss(X, g, h0), G, v), (dG * v).sum(), rtol=1e-7, atol=1e-8)
    assert (dG[np.isneginf(G)] == 0).all()
    v = rng.normal(size=h0.shape)
    assert np.isclose(slope(lambda h: loss(X, G, h), h0, v), (dh0 * v).sum(), rtol=1e-7, atol=1e-8)


def test_gated_forgets_what_is_not_finite():
    X, G = np.ones((1, 4, 2)), np.full((1, 4, 2), -0.5)
    X[0, 0] = [np.nan, np.inf]
    G[0, 2] = -np.inf
    Z = ref.gated(X, G, np.zeros((1, 2)))
    assert not np.isfinite(Z[0, :2]).any() and np.array_equal(Z[0, 2], [1.0, 1.0])


def test_rmsnorm_gradients():
    rng = np.random.default_rng(4)
    x, w, dY, dR = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))

    def loss(x, w):
        y, r = ref.rmsnorm(x, w, None, 1e-3)
        return (y * dY).sum() + (r * dR).sum()

    dx, dw = ref.rmsnorm_bwd(x, w, dY, dR, 1e-3)
    v = rng.normal(size=x.shape)
    assert np.isclose(slope(lambda t: loss(t, w), x, v), (dx * v).sum(), rtol=1e-7)
    v = rng.normal(size=w.shape)
    assert np.isclose(slope(lambda t: loss(x, t), w, v), (dw * v).sum(), rtol=1e-7)


def test_within_counts_one_rounding():
    assert ref.within(1.0 + 2.0 ** -8, 1.0, 0.0, "bf16")[0]
    assert not ref.within(1.0 + 2.0 ** -7, 1.0, 0.0, "bf16")[0]
    assert not ref.within(np.array([np.nan]), np.array([1.0]), 1.0, "f32")[0]
    assert not ref.within(np.array([np.inf]), np.array([-np.inf]), 1.0, "f32")[0]
