"""Plain fp64 forms of the gated delta rule, group norm with an activation and dropout, with the
error bounds that the tests hold the kernels to.

U is half a step of fp32 (2^-24), HALF[io] half a step of the I/O type relative to the value."""
import math

import numpy as np

from block_ref import HALF, U, within  # noqa: F401


def delta(K, Q, V, eta, g, W0):
    """(Z, W_T, states before each token, u) of [N, T, d] arrays, one head of keys for each of
    values; eta, g: [N, T], W0: [N, dv, dk]."""
    K, Q, V, eta, g, W = (np.asarray(x, np.float64) for x in (K, Q, V, eta, g, W0))
    N, T, _ = K.shape
    Z, u = np.empty_like(V), np.empty_like(V)
    before = np.empty((T,) + W.shape)
    for t in range(T):
        before[t] = W
        W = np.where(g[:, t] <= -1e30, 0.0, np.exp(g[:, t]))[:, None, None] * W
        u[:, t] = V[:, t] - np.einsum("nvk,nk->nv", W, K[:, t])
        W = W + np.einsum("nv,nk->nvk", eta[:, t, None] * u[:, t], K[:, t])
        Z[:, t] = np.einsum("nvk,nk->nv", W, Q[:, t])
    return Z, W, before, u


def delta_bwd(K, Q, V, eta, g, W0, dZ, dW):
    """(dK, dQ, dV, deta, dg, dW0) in fp64."""
    K, Q, V, eta, g, W0, dZ, D = (np.asarray(x, np.float64) for x in (K, Q, V, eta, g, W0, dZ, dW))
    _, _, before, u = delta(K, Q, V, eta, g, W0)
    dK, dQ, dV = np.empty_like(K), np.empty_like(Q), np.empty_like(V)
    deta, dg = np.empty_like(eta), np.empty_like(g)
    for t in range(K.shape[1] - 1, -1, -1):
        a = np.where(g[:, t] <= -1e30, 0.0, np.exp(g[:, t]))[:, None, None]
        k, q, w = K[:, t], Q[:, t], eta[:, t, None] * u[:, t]
        kept = a * before[t]
        now = kept + np.einsum("nv,nk->nvk", w, k)
        D = D + np.einsum("nv,nk->nvk", dZ[:, t], q)
        dQ[:, t] = np.einsum("nvk,nv->nk", now, dZ[:, t])
        dw = np.einsum("nvk,nk->nv", D, k)
        deta[:, t] = (dw * u[:, t]).sum(1)
        dV[:, t] = eta[:, t, None] * dw
        dK[:, t] = np.einsum("nvk,nv->nk", D, w) - np.einsum("nvk,nv->nk", kept, dV[:, t])
        D = D - np.einsum("nv,nk->nvk", dV[:, t], k)
        dg[:, t] = (D * kept).sum((1, 2))
        D = a * D
    return dK, dQ, dV, deta, dg, D


def delta_rel(T, dk, dv):
    """Error of an output relative to the largest of its (batch, head), before its own rounding.

    An output passes through products over dk features, dv columns and three times 64 tokens for
    each chunk, their operands good to 2^-24 (three bf16 parts), summed in fp32: 4 n roundings of U
    each, n = dk + dv + 192, of no common sign, so sqrt(4 n) U, and 6 times that for the largest of
    some 10^5 values (6 standard deviations: 2e-9 each).  Keys of at most unit length with
    0 <= eta <= 1 and g <= 0 do not enlarge what came before, so chunks add up alike."""
    return 6 * math.sqrt(4 * (dk + dv + 192) * (1 + T // 64)) * U


# of a bf16 Z: products of two parts by two leave 2^-16 of each term at most (2^-17 for an operand's
# third part, 2^-18 for the product of the second ones), a state, u and P each once
Z_BF16 = 3 * 2.0 ** -16


def groups(X, G):
    """[N, S, C] as [N, G, S C / G]."""
    N, S, C = X.shape
    return X.reshape(N, S, G, C // G).transpose(0, 2, 1, 3).reshape(N, G, -1)


def ungroup(x, shape, G):
    N, S, C = shape
    return x.reshape(N, G, S, C // G).transpose(0, 2, 1, 3).reshape(shape)


def _erf(v):
    return np.vectorize(math.erf, otypes=[np.float64])(v)


def activation(v, act):
    """(value, derivative)"""
    with np.errstate(over="ignore"):
        if act == "silu":
            s = 1.0 / (1.0 + np.exp(-v))
            return v * s, s + v * s * (1.0 - s)
        if act == "gelu":
            p = 0.5 * (1.0 + _erf(v / math.sqrt(2.0)))
            return v * p, p + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    return v, np.ones_like(v)


def groupnorm(X, G, w, b, eps, act):
    """(y, mean, rstd, bound of y, of mean, relative bound of rstd) in fp64.

    Sums of m values of which each passes through at most m / 64 + 40 additions (a thread's own and
    the joins): c U of the mean of |x| for the mean, c + 8 relative for the variance, and half of
    that for rstd; (x - mean) takes the mean's error and one rounding, the affine part two, and the
    activation (slope at most 1.13) 8 + 2 |v| U of its value (exp of -v: its argument's rounding)."""
    X = np.asarray(X, np.float64)
    N, S, C = X.shape
    x = groups(X, G)
    mean = x.mean(2)
    d = x - mean[..., None]
    rstd = 1.0 / np.sqrt((d * d).mean(2) + eps)
    c = (x.shape[2] / 64 + 40) * U
    em = c * np.abs(x).mean(2)
    rel = 0.5 * (2 * c + 8 * U) + 4 * U + (em * rstd) ** 2
    n = ungroup(d * rstd[..., None], X.shape, G)
    en = ungroup((em[..., None] + U * np.abs(d)) * rstd[..., None], X.shape, G) + np.abs(n) * (
        ungroup(np.broadcast_to(rel[..., None], x.shape), X.shape, G) + U)
    w = np.ones(C) if w is None else np.asarray(w, np.float64)
    b = np.zeros(C) if b is None else np.asarray(b, np.float64)
    v = n * w + b
    ev = en * np.abs(w) + 2 * U * (np.abs(n * w) + np.abs(v))
    y = activation(v, act)[0]
    return y, mean, rstd, 1.13 * ev + (8 + 2 * np.abs(v)) * U * np.abs(y) + 2 * U * np.abs(v), em, rel


def groupnorm_bwd(X, G, w, b, dY, mean, rstd, act):
    """(dx, dweight, dbias) in fp64 and their bounds: dv takes the derivative's error (slope at most
    1 in v, whose own roundings are 4 U (|n w| + |v|); 16 U of exp and quotient), the two means c U
    of the means of the absolute values, and dx three roundings of its parts; the sums over N S rows
    at most N S + 24 additions."""
    X, dY, mean, rstd = (np.asarray(t, np.float64) for t in (X, dY, mean, rstd))
    N, S, C = X.shape
    x = groups(X, G)
    r = rstd[..., None]
    n = ungroup((x - mean[..., None]) * r, X.shape, G)
    w = np.ones(C) if w is None else np.asarray(w, np.float64)
    b = np.zeros(C) if b is None else np.asarray(b, np.float64)
    v = n * w + b
    dv = dY * activation(v, act)[1]
    u = dv * w
    m = lambda t: ungroup(np.broadcast_to(groups(t, G).mean(2, keepdims=True), x.shape), X.shape, G)  # noqa: E731
    rr = ungroup(np.broadcast_to(r, x.shape), X.shape, G)
    dx = rr * (u - m(u) - n * m(u * n))
    edv = np.abs(dY) * (16 * U * (1 + np.abs(v)) + 4 * U * (np.abs(n * w) + np.abs(v)))
    eu = edv * np.abs(w) + U * np.abs(u)
    c = (x.shape[2] / 64 + 40) * U
    e1 = m(eu) + c * m(np.abs(u))
    e2 = m(eu * np.abs(n)) + (c + 4 * U) * m(np.abs(u * n))
    edx = rr * (eu + e1 + np.abs(n) * e2 + 6 * U * (np.abs(u) + m(np.abs(u)) + np.abs(n) * m(np.abs(u * n))))
    k = (N * S + 24) * U
    rows = lambda t: t.reshape(-1, C).sum(0)  # noqa: E731
    return (dx, rows(dv * n), rows(dv)), (edx, rows(edv * np.abs(n) + (k + 4 * U) * np.abs(dv * n)),
                                          rows(edv + k * np.abs(dv)))


def philox(counter, key):
    """Philox 4x32 of 10 rounds: counter [n, 4] and key (two words) to [n, 4], all uint64 below 2^32."""
    x = [np.asarray(counter[:, i], np.uint64) for i in range(4)]
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for r in range(10):
        k = [np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)]
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> s) ^ x[1] ^ k[0], b & low, (a >> s) ^ x[3] ^ k[1], a & low]
    return np.stack(x, 1)


def keep_mask(n, p, seed, first):
    """Which of n elements dropout keeps."""
    at = [(first + i) % (1 << 64) for i in range((n + 3) // 4)]
    counter = np.array([[a & 0xFFFFFFFF, a >> 32, 0, 0] for a in at], np.uint64).reshape(-1, 4)
    key = (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)
    return philox(counter, key).reshape(-1)[:n] >= np.uint64(round(p * 4294967296.0))
