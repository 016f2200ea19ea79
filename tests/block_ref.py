"""Plain fp64 forms of the operators around the scan (gated recurrence, RMS norm, gradient
clipping) with the error bounds that the tests hold the kernels to.

The bounds are worst-case counts of roundings.  U is half a step of fp32 (2^-24), HALF[io] half a
step of the I/O type relative to the value (one rounding of an output)."""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
E4M3_MAX = 448.0


def decay(a, shut, h):
    """a h, where a shut gate leaves nothing whatever h is."""
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(shut, 0.0, a * h)


def gated(X, G, h0):
    """All states of h_t = exp(g_t) h_{t-1} + x_t; X, G: [N, T, d], h0: [N, d]."""
    X, G = X.astype(np.float64), G.astype(np.float64)
    a, shut = np.exp(G), np.isneginf(G)
    h, Z = h0.astype(np.float64), np.empty_like(X)
    for t in range(X.shape[1]):
        h = decay(a[:, t], shut[:, t], h) + X[:, t]
        Z[:, t] = h
    return Z


def gated_bound(X, G, h0):
    """Elementwise bound of the fp32 evaluation's error, before the output's rounding.

    One step h = fl(a h) + x carries on the error of h times a and adds the gate's own error (the
    product g log2(e) rounded: at most 1.5 |g| U; exp2: 2 U) and two roundings, together
    (4 + 3 |g|) U of the majorant H_t = exp(g_t) H_{t-1} + |x_t|.  Where a state enters a run of
    up to 256 tokens by the exponential of their summed g, that sum's error is at most 256 U |sum|,
    and |sum| exp(sum) <= 0.37: 128 U of the largest majorant, once for every run: the runs' errors
    decay with the states, so they add up as the steps' do, through the same recurrence."""
    G = G.astype(np.float64)
    H = gated(np.abs(X), G, np.abs(h0))
    big = np.nanmax(np.where(np.isfinite(H), H, 0.0), axis=1, keepdims=True)
    step = (4 + 3 * np.where(np.isneginf(G), 0.0, np.abs(G))) * U * H
    return gated(step, G, np.zeros_like(h0)) + 128 * U * big * (1 + X.shape[1] // 256)


def gated_bwd(G, Z, h0, dZ, dhT):
    """(dX, dG, dh0) in fp64."""
    G, Z, lam = G.astype(np.float64), Z.astype(np.float64), dZ.astype(np.float64).copy()
    a, shut = np.exp(G), np.isneginf(G)
    carry = dhT.astype(np.float64)
    dG = np.empty_like(lam)
    for t in range(G.shape[1] - 1, -1, -1):
        lam[:, t] += carry
        carry = decay(a[:, t], shut[:, t], lam[:, t])
        before = Z[:, t - 1] if t else h0.astype(np.float64)
        with np.errstate(invalid="ignore"):
            dG[:, t] = np.where(shut[:, t], 0.0, carry * before)
    return lam, dG, carry


def gated_bwd_bound(G, Z, h0, dZ, dhT):
    """Bounds of (dX, dG, dh0) before the outputs' rounding: lambda is the same recurrence from the
    other end; dg = exp(g) lambda h takes lambda's error and (6 + 3 |g|) U of its own."""
    N, T, d = G.shape
    G = G.astype(np.float64)
    shift = np.concatenate([G[:, 1:], np.zeros((N, 1, d))], 1)
    e = gated_bound(dZ[:, ::-1], shift[:, ::-1], dhT)[:, ::-1]
    a, shut = np.exp(G), np.isneginf(G)
    lam, dG, dh0 = gated_bwd(G, Z, h0, dZ, dhT)
    before = np.concatenate([h0[:, None].astype(np.float64), Z[:, :-1].astype(np.float64)], 1)
    own = (6 + 3 * np.where(shut, 0.0, np.abs(G))) * U
    edg = np.where(shut, 0.0, a * e * np.abs(before) + own * np.abs(dG))
    edh = np.where(shut[:, 0], 0.0, a[:, 0] * e[:, 0] + own[:, 0] * np.abs(dh0))
    return e, edg, edh


def rmsnorm(X, w, res, eps):
    """(y, r) in fp64."""
    r = X.astype(np.float64) + (0.0 if res is None else res.astype(np.float64))
    k = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return r * k * (1.0 if w is None else w.astype(np.float64)), r


def rms_rel(D):
    """Relative error of k = 1 / sqrt(mean(r^2) + eps) in fp32, in units of U: a sum of positive terms
    in which each passes through at most D / 64 + 12 additions (half of that reaches k), r's own
    rounding twice, the division by D, the addition of eps, and a reciprocal square root good to
    2 steps (4 U)."""
    return 0.5 * (D / 64 + 16) + 6


def rmsnorm_bwd(R, w, dY, dR, eps):
    """(dx, dweight) in fp64."""
    R, dY = R.astype(np.float64), dY.astype(np.float64)
    k = 1.0 / np.sqrt((R * R).mean(-1, keepdims=True) + eps)
    n = R * k
    u = dY * (1.0 if w is None else w.astype(np.float64))
    dx = k * (u - n * (u * n).mean(-1, keepdims=True))
    if dR is not None:
        dx = dx + dR.astype(np.float64)
    return dx, (dY * n).sum(0)


def rmsnorm_bwd_bound(R, w, dY, dR, eps):
    """Bounds of (dx, dweight) before the output's rounding.  mean(u n) is a sum of D terms of either
    sign: at most (D / 64 + 16) U of the mean of |u n|, and k's error; dx = k (u - n m) + dr: three
    roundings each; dweight: at most rows U of the sum of |dy n| (any order of additions), and k's
    error and two roundings of each term."""
    R, dY = R.astype(np.float64), dY.astype(np.float64)
    rows, D = R.shape
    k = 1.0 / np.sqrt((R * R).mean(-1, keepdims=True) + eps)
    n = np.abs(R * k)
    u = np.abs(dY * (1.0 if w is None else w.astype(np.float64)))
    m = (u * n).mean(-1, keepdims=True)
    rel = rms_rel(D)
    edx = k * (u * (rel + 6) + n * m * (3 * rel + D / 64 + 24)) * U
    if dR is not None:
        edx = edx + 2 * U * (np.abs(dR.astype(np.float64)) + k * (u + n * m))
    edw = (rows + rel + 4) * U * (np.abs(dY) * n).sum(0)
    return edx, edw


def clip(grads, max_norm, eps):
    """(outs, norm) in fp64."""
    norm = np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    f = min(1.0, max_norm / (norm + eps))
    return [g.astype(np.float64) * f for g in grads], norm


def within(got, ref, bound, io):
    """(ok, worst ratio of the error to what is allowed): |got - ref| <= bound + half a step of the
    output's type; what is not finite has to be so alike."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    fine = np.isfinite(ref)
    if not np.array_equal(np.isnan(got), np.isnan(ref)):
        return False, np.inf
    inf = ~fine & ~np.isnan(ref)
    if not np.array_equal(got[inf], ref[inf]):
        return False, np.inf
    room = np.broadcast_to(bound, ref.shape)[fine] * (1 + HALF[io]) + HALF[io] * np.abs(ref[fine]) + 1e-38
    err = np.abs(got[fine] - ref[fine])
    worst = float((err / room).max()) if err.size else 0.0
    return worst <= 1.0, worst
