"""Cases of the gated delta rule and of the block around it, in their plain form and through the library.

  delta      the gated delta rule, a fast-weight state W [dv, dk] per (batch, head) that takes one gradient step
             per token and decays:
                 u_t = v_t - exp(g_t) W_{t-1} k_t,   W_t = exp(g_t) W_{t-1} + eta_t u_t k_t^T,   z_t = W_t q_t,
             over whole sequences ("fwd"), its gradients ("bwd") and the continuation by a few tokens ("step").
             g_t <= 0 is the logarithm of the decay; -inf forgets everything before, which is how documents packed
             in one row start anew; eta_t = 0 with g_t = 0 carries the state through padding. Groups of heads may
             share keys and queries, and tokens lie as [B, H, T, d] or as [B, T, H, d].
  groupnorm  the norm over each group of channels of a channels-last tensor [N, S, C], scaled, shifted and passed
             through an activation; with S = 1 it is the norm of every head's output of every token. Forward, with
             the statistics ("fwd"), and backward ("bwd").
  dropout    x / (1 - p) or 0 by a counter-based generator (Philox 4x32 of 10 rounds, 32 bits an element), with the
             residual's addition; the gradient is the same call, so no mask is stored.

`own` chooses between the plain torch form (elementary operations in 32 bits, rounded once at the end) and
the library's kernels; both take what prepare() gives.
"""
import math

import numpy as np
import torch

own = False

_IO = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_EPS = 1e-5
_FORGET = -1e30
_C = 64                                   # tokens of a chunk in the plain form


def listed():
    return [
        # one decoded token of 8 x 12 heads: a call whose latency counts
        {"name": "delta step 8x12x1 d64", "op": "delta", "form": "step", "B": 8, "H": 12, "share": 1, "T": 1, "dk": 64,
         "dv": 64, "io": "bf16", "layout": "bhtd", "resets": 0, "pad": 0, "start": True},
        # one decoded token of a large serving batch: the states are read and written once
        {"name": "delta step 256x12x1 d64", "op": "delta", "form": "step", "B": 256, "H": 12, "share": 1, "T": 1,
         "dk": 64, "dv": 64, "io": "bf16", "layout": "bhtd", "resets": 0, "pad": 0, "start": True},
        # a training or prefill batch at the many-head configuration
        {"name": "delta fwd 8x12x2048 d64", "op": "delta", "form": "fwd", "B": 8, "H": 12, "share": 1, "T": 2048,
         "dk": 64, "dv": 64, "io": "bf16", "layout": "bhtd", "resets": 0, "pad": 0, "start": True},
        # one long document: few heads, so the time axis has to be shared out
        {"name": "delta fwd 1x32x32768 d64", "op": "delta", "form": "fwd", "B": 1, "H": 32, "share": 1, "T": 32768,
         "dk": 64, "dv": 64, "io": "bf16", "layout": "bhtd", "resets": 0, "pad": 0, "start": True},
        # fp32, odd length and widths, packed documents (resets) and a padded tail, no initial state, tokens first
        {"name": "delta fwd f32 3x5x1001 50-83", "op": "delta", "form": "fwd", "B": 3, "H": 5, "share": 1, "T": 1001,
         "dk": 50, "dv": 83, "io": "f32", "layout": "bthd", "resets": 5, "pad": 100, "start": False},
        # the training step's backward pass at the many-head configuration
        {"name": "delta bwd 8x12x2048 d64", "op": "delta", "form": "bwd", "B": 8, "H": 12, "share": 1, "T": 2048,
         "dk": 64, "dv": 64, "io": "bf16", "layout": "bhtd", "resets": 4, "pad": 0, "start": True},
        # the backward pass with wide heads, two of them for each head of keys and queries
        {"name": "delta bwd 2x16x4096 d128", "op": "delta", "form": "bwd", "B": 2, "H": 16, "share": 2, "T": 4096,
         "dk": 128, "dv": 128, "io": "bf16", "layout": "bthd", "resets": 0, "pad": 0, "start": True},
        # the norm of 32 heads of 64 for every token of 8 x 2048
        {"name": "groupnorm fwd 16384x1x2048", "op": "groupnorm", "form": "fwd", "N": 16384, "S": 1, "C": 2048,
         "G": 32, "io": "bf16", "act": "silu", "affine": True},
        # whole slabs of 64 x 64 places, 20 channels a group
        {"name": "groupnorm fwd 8x4096x640", "op": "groupnorm", "form": "fwd", "N": 8, "S": 4096, "C": 640,
         "G": 32, "io": "bf16", "act": "silu", "affine": True},
        # the token norm's backward pass in training
        {"name": "groupnorm bwd 16384x1x2048", "op": "groupnorm", "form": "bwd", "N": 16384, "S": 1, "C": 2048,
         "G": 32, "io": "bf16", "act": "silu", "affine": True},
        # a block's output on its way into the residual stream, 8 x 2048 tokens of 2048 features
        {"name": "dropout 33554432 residual", "op": "dropout", "n": 33554432, "io": "bf16", "p": 0.1,
         "residual": True},
        # an odd number of fp32 values, half of them dropped
        {"name": "dropout f32 1000003", "op": "dropout", "n": 1000003, "io": "f32", "p": 0.5, "residual": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "groupnorm", "groupnorm", "dropout"])
    io = rng.choice(["bf16", "f32"])
    if op == "delta":
        form = rng.choice(["fwd", "fwd", "bwd", "bwd", "step"])
        share = rng.choice([1, 1, 2, 4])
        B, H = _log(rng, 1, 16), share * _log(rng, 1, 32 // share)
        dk, dv = rng.choice([16, 32, 50, 64, 64, 96, 128]), rng.choice([16, 32, 64, 64, 83, 128, 200, 256])
        most = 4294967296 if form != "bwd" else 2147483648
        T = rng.randint(1, 8) if form == "step" else _log(rng, 2, 32768)
        T = max(1, min(T, most // (B * H * dk * dv)))
        return {"op": op, "form": form, "B": B, "H": H, "share": share, "T": T, "dk": dk, "dv": dv, "io": io,
                "layout": rng.choice(["bhtd", "bthd"]), "resets": rng.choice([0, 3, 17]),
                "pad": rng.choice([0, T // 5]), "start": rng.random() < 0.5}
    most = 33554432 if io == "bf16" else 16777216
    if op == "groupnorm":
        G = rng.choice([1, 4, 8, 32])
        C = G * rng.choice([1, 3, 8, 16, 20, 64, 80, 128])
        N = _log(rng, 1, 65536) if rng.random() < 0.5 else _log(rng, 1, 64)
        S = 1 if N > 64 else rng.choice([1, 49, 1024, 4096, 9999, 16384])
        N = max(1, min(N, most // (S * C)))
        return {"op": op, "form": rng.choice(["fwd", "bwd"]), "N": N, "S": S, "C": C, "G": G, "io": io,
                "act": rng.choice(["none", "silu", "gelu"]), "affine": rng.random() < 0.8}
    return {"op": op, "n": _log(rng, 1, most), "io": io, "p": rng.choice([0.0, 0.1, 0.25, 0.9]),
            "residual": rng.random() < 0.5}


def _heads(t, layout):
    """Between [B, H, T, ...] and the layout of the case's token tensors."""
    return t if layout == "bhtd" else t.transpose(1, 2).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    s = {"case": case}
    io = _IO[case["io"]]
    if case["op"] == "delta":
        B, H, T, dk, dv, lay = (case[k] for k in ("B", "H", "T", "dk", "dv", "layout"))
        K, Q = normal(B, H // case["share"], T, dk), normal(B, H // case["share"], T, dk)
        # unit keys and queries, as such layers norm them; step sizes around a half; decays of a trained layer
        K, Q = K / K.norm(dim=3, keepdim=True), Q / Q.norm(dim=3, keepdim=True)
        V, eta = normal(B, H, T, dv), torch.sigmoid(normal(B, H, T))
        g = torch.nn.functional.logsigmoid(normal(B, H, T) + 4.0)
        if case["resets"]:
            at = torch.randint(0, T, (case["resets"],), device=dev, generator=gen)
            g[:, :, at] = -math.inf
        if case["pad"]:
            g[-1:, :, T - case["pad"]:] = 0.0
            eta[-1:, :, T - case["pad"]:] = 0.0
        for name, t in (("K", K), ("Q", Q), ("V", V)):
            s[name] = _heads(t.to(io), lay)
        s["eta"], s["g"] = _heads(eta, lay), _heads(g, lay)
        s["W"] = 0.3 * normal(B, H, dv, dk) if case["start"] else None
        if case["form"] == "step" and s["W"] is None:
            s["W"] = torch.zeros(B, H, dv, dk, device=dev)
        if case["form"] == "bwd":
            s["dZ"] = _heads(normal(B, H, T, dv).to(io), lay)
            s["dW"] = normal(B, H, dv, dk) if case["start"] else None
    elif case["op"] == "groupnorm":
        N, S, C, G = (case[k] for k in "NSCG")
        # channels of different means and spreads
        s["X"] = (normal(N, S, C) * (0.5 + torch.rand(C, device=dev, generator=gen)) + 0.5 * normal(C)).to(io)
        s["w"] = 1.0 + 0.1 * normal(C) if case["affine"] else None
        s["b"] = 0.1 * normal(C) if case["affine"] else None
        if case["form"] == "bwd":
            x = s["X"].float().view(N, S, G, C // G)
            s["mean"] = x.mean((1, 3))
            s["rstd"] = 1.0 / torch.sqrt((x - s["mean"][:, None, :, None]).square().mean((1, 3)) + _EPS)
            s["dY"] = normal(N, S, C).to(io)
    else:
        s["X"] = normal(case["n"]).to(io)
        s["res"] = (2.0 * normal(case["n"])).to(io) if case["residual"] else None
        # the generator's seed and the first counter of this call
        s["rng"] = torch.tensor([0x1234567890ABCDE ^ (int(seed) * 2654435761), 4000000000 + int(seed) * 8388608],
                                dtype=torch.int64, device=dev)
    return s


def _chunked(s, names):
    """The token tensors as [B H, chunks, 64, d] in fp32, one head of keys for every head of values, the last chunk
    filled with tokens that change nothing."""
    c, out = s["case"], []
    for name in names:
        t = s[name].float()
        t = t.transpose(1, 2) if c["layout"] == "bthd" else t
        if t.shape[1] < c["H"]:
            t = t.repeat_interleave(c["share"], 1)
        fill = -c["T"] % _C
        t = torch.cat([t, t.new_zeros(t.shape[:2] + (fill,) + t.shape[3:])], 2)
        out.append(t.reshape(c["B"] * c["H"], -1, _C, *t.shape[3:]).contiguous())
    return out


def _unchunked(s, t):
    """From [B H, chunks, 64, d] back to the layout of the case."""
    c = s["case"]
    t = t.reshape(c["B"], c["H"], -1, *t.shape[3:])[:, :, :c["T"]]
    return t.transpose(1, 2).contiguous() if c["layout"] == "bthd" else t.contiguous()


def _decays(g):
    """E [.., t, s] = product of the decays after s up to t (s <= t), each token's from the chunk's start, and from
    each token to the chunk's end; sums of logarithms in 64 bits."""
    cut = g <= _FORGET
    G = torch.where(cut, 0.0, g.double()).cumsum(2)
    n = cut.cumsum(2)
    E = torch.exp(G[..., :, None] - G[..., None, :]) * (n[..., :, None] == n[..., None, :])
    return torch.tril(E).float(), (torch.exp(G) * (n == 0)).float()[..., None], E[..., -1, :].float()[..., None]


def _inverse(N):
    """(I - N)^-1 of strictly lower triangular N of 64 rows: (I + N) (I + N^2) (I + N^4) ..."""
    eye = torch.eye(_C, device=N.device)
    out, power = eye + N, N @ N
    for _ in range(5):
        out, power = out + out @ power, power @ power
    return out


def _delta_states(s):
    """The forward pass by chunks: U = (I + L eta)^-1 (V - start K W^T) holds what each token writes, W the states
    at the chunks' starts and at the end."""
    c = s["case"]
    K, Q, V, eta, g = _chunked(s, ("K", "Q", "V", "eta", "g"))
    eta = eta[..., None]
    E, start, end = _decays(g)
    L = torch.tril(E * (K @ K.transpose(2, 3)), -1)
    inv = _inverse(-L * eta.transpose(2, 3))
    W = torch.zeros(K.shape[0], c["dk"], c["dv"], device=K.device) if s["W"] is None \
        else s["W"].reshape(-1, c["dv"], c["dk"]).transpose(1, 2)
    states, U = [W], []
    for n in range(K.shape[1]):
        U.append(inv[:, n] @ (V[:, n] - start[:, n] * (K[:, n] @ W)))
        W = start[:, n, -1:] * W + K[:, n].transpose(1, 2) @ (end[:, n] * eta[:, n] * U[-1])
        states.append(W)
    return K, Q, eta, E, start, end, L, inv, torch.stack(states, 1), torch.stack(U, 1)


def _delta(s):
    c, io = s["case"], s["K"].dtype
    K, Q, eta, E, start, end, L, inv, W, U = _delta_states(s)
    P = E * (Q @ K.transpose(2, 3))
    last = W[:, -1].transpose(1, 2).reshape(c["B"], c["H"], c["dv"], c["dk"])
    if c["form"] != "bwd":
        Z = _unchunked(s, start * (Q @ W[:, :-1]) + P @ (eta * U)).to(io)
        if c["form"] == "step":
            return Z, s["W"].copy_(last)
        return Z, last.contiguous()
    (dZ,) = _chunked(s, ("dZ",))
    D = torch.zeros_like(W[:, 0]) if s["dW"] is None else s["dW"].reshape(-1, c["dv"], c["dk"]).transpose(1, 2)
    Ds, dVs, Fs = [D], [], []
    for n in range(K.shape[1] - 1, -1, -1):
        dU = P[:, n].transpose(1, 2) @ dZ[:, n] + end[:, n] * (K[:, n] @ D)
        dV = inv[:, n].transpose(1, 2) @ (eta[:, n] * dU)
        Fs.append(dU - L[:, n].transpose(1, 2) @ dV)
        dVs.append(dV)
        D = start[:, n, -1:] * D + Q[:, n].transpose(1, 2) @ (start[:, n] * dZ[:, n]) \
            - K[:, n].transpose(1, 2) @ (start[:, n] * dV)
        Ds.append(D)
    D, dV, F = (torch.stack(t[::-1], 1) for t in (Ds, dVs, Fs))
    W0, DT, u = W[:, :-1], D[:, 1:], eta * U
    dP = torch.tril(dZ @ u.transpose(2, 3)) * E
    dL = -torch.tril(dV @ u.transpose(2, 3), -1) * E
    read, kept, written = start * (dZ @ W0.transpose(2, 3)), start * (dV @ W0.transpose(2, 3)), \
        end * (u @ DT.transpose(2, 3))
    dQ = read + dP @ K
    dK = dP.transpose(2, 3) @ Q + dL @ K + dL.transpose(2, 3) @ K + written - kept
    # a decay g_t lies between every token from t on and all that was written before t: the products over
    # these pairs, summed in 64 bits
    pairs = torch.tril(dP * (Q @ K.transpose(2, 3)) + dL * (K @ K.transpose(2, 3)), -1).double()
    across = pairs.cumsum(3).flip(2).cumsum(2).flip(2)
    dg = torch.cat([torch.zeros_like(across[:, :, :1, 0]), across.diagonal(-1, 2, 3)], 2)
    reads = (read * Q - kept * K).double().sum(3)
    writes = (written * K).double().sum(3)
    dg = dg + reads.flip(2).cumsum(2).flip(2) + writes.cumsum(2) - writes \
        + (start[:, :, -1, 0].double() * (DT * W0).double().sum((2, 3)))[..., None]
    dg = torch.where(_chunked(s, ("g",))[0] <= _FORGET, 0.0, dg)
    dQ, dK = _unchunked(s, dQ), _unchunked(s, dK)
    if c["share"] > 1:
        h = 1 if c["layout"] == "bhtd" else 2
        dQ, dK = (t.unflatten(h, (-1, c["share"])).sum(h + 1) for t in (dQ, dK))
    dW0 = D[:, 0].transpose(1, 2).reshape(c["B"], c["H"], c["dv"], c["dk"]).contiguous()
    return dK.to(io), dQ.to(io), _unchunked(s, dV).to(io), _unchunked(s, (F * U).sum(3)), \
        _unchunked(s, dg).float(), dW0


def _activation(v, act):
    """The activation's value and its derivative."""
    if act == "silu":
        y = torch.sigmoid(v)
        return v * y, y * (1.0 + v * (1.0 - y))
    if act == "gelu":
        y = 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
        return v * y, y + v * torch.exp(-0.5 * v * v) * math.sqrt(0.5 / math.pi)
    return v, torch.ones_like(v)


def _groupnorm(s):
    c, io = s["case"], s["X"].dtype
    N, S, C, G = (c[k] for k in "NSCG")
    x = s["X"].float().view(N, S, G, C // G)
    w = s["w"] if s["w"] is not None else torch.ones(C, device=x.device)
    b = s["b"] if s["b"] is not None else torch.zeros(C, device=x.device)
    w, b = w.view(G, C // G), b.view(G, C // G)
    if c["form"] == "fwd":
        mean = x.mean((1, 3))
        rstd = 1.0 / torch.sqrt((x - mean[:, None, :, None]).square().mean((1, 3)) + _EPS)
        n = (x - mean[:, None, :, None]) * rstd[:, None, :, None]
        return _activation(n * w + b, c["act"])[0].to(io).view(N, S, C), mean, rstd
    n = (x - s["mean"][:, None, :, None]) * s["rstd"][:, None, :, None]
    dv = s["dY"].float().view(N, S, G, C // G) * _activation(n * w + b, c["act"])[1]
    u = dv * w
    dx = s["rstd"][:, None, :, None] * (u - u.mean((1, 3), keepdim=True) - n * (u * n).mean((1, 3), keepdim=True))
    return dx.to(io).view(N, S, C), (dv * n).sum((0, 1)).view(C), dv.sum((0, 1)).view(C)


def _multiply(a, b):
    """The two 32-bit halves of a times b, both below 2^32."""
    low, high = a * (b & 0xFFFF), a * (b >> 16)
    return (high + (low >> 16)) >> 16, ((high << 16) + low) & 0xFFFFFFFF


def _random(rng, n):
    """n 32-bit numbers: element i has word i % 4 of the block whose counter is first + i / 4."""
    at = rng[1] + torch.arange((n + 3) // 4, device=rng.device)
    c0, c1 = at & 0xFFFFFFFF, (at >> 32) & 0xFFFFFFFF
    c2, c3 = torch.zeros_like(at), torch.zeros_like(at)
    k0, k1 = rng[0] & 0xFFFFFFFF, (rng[0] >> 32) & 0xFFFFFFFF
    for _ in range(10):
        (h0, l0), (h1, l1) = _multiply(0xD2511F53, c0), _multiply(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack([c0, c1, c2, c3], 1).reshape(-1)[:n]


def _dropout(s):
    c, io = s["case"], s["X"].dtype
    keep = _random(s["rng"], c["n"]) >= int(round(c["p"] * 4294967296.0))
    y = torch.where(keep, s["X"].float() * (1.0 / (1.0 - c["p"])), torch.zeros((), device=keep.device))
    return (y + s["res"].float() if s["res"] is not None else y).to(io)


def _library(s):
    from test_sequence_layers_ttt_amd import ttt
    c = s["case"]
    if c["op"] == "delta":
        layout = ttt.LAYOUT_BHTD if c["layout"] == "bhtd" else ttt.LAYOUT_BTHD
        if c["form"] == "step":
            return ttt.delta_step(s["K"], s["Q"], s["V"], s["eta"], s["g"], s["W"], layout=layout), s["W"]
        if c["form"] == "fwd":
            return ttt.delta_fwd(s["K"], s["Q"], s["V"], s["eta"], s["g"], s["W"], layout=layout)
        return ttt.delta_bwd(s["K"], s["Q"], s["V"], s["eta"], s["g"], s["W"], s["dZ"], s["dW"], layout=layout)
    if c["op"] == "groupnorm":
        act = {"none": ttt.ACT_NONE, "silu": ttt.ACT_SILU, "gelu": ttt.ACT_GELU}[c["act"]]
        if c["form"] == "fwd":
            return ttt.groupnorm_fwd(s["X"], c["G"], s["w"], s["b"], _EPS, act)
        return ttt.groupnorm_bwd(s["X"], c["G"], s["w"], s["b"], s["dY"], s["mean"], s["rstd"], act)
    return ttt.dropout(s["X"], c["p"], s["rng"], s["res"])


def run(state):
    if own:
        return _library(state)
    op = state["case"]["op"]
    out = _delta(state) if op == "delta" else _groupnorm(state) if op == "groupnorm" else _dropout(state)
    if op == "groupnorm" and state["case"]["form"] == "bwd" and not state["case"]["affine"]:
        return out[0], None, None
    return out


def work(case):
    e = _SIZE[case["io"]]
    if case["op"] == "delta":
        heads = case["B"] * case["H"]
        n, dk, dv, state = heads * case["T"], case["dk"], case["dv"], 4 * heads * case["dk"] * case["dv"]
        keys, values, gates = 2 * e * dk * n // case["share"], e * dv * n, 8 * n
        if case["form"] == "bwd":  # K, Q, V, dZ, gates in, dK, dQ, dV, their gradients out; W0 and dW_T in, dW0 out
            return {"bytes": 2 * keys + 3 * values + 2 * gates + state * (3 if case["start"] else 1),
                    "flops": 18 * n * dk * dv}
        # K, Q, V and gates in, Z out; the last state out, the first in where there is one
        return {"bytes": keys + 2 * values + gates + state * (2 if case["start"] or case["form"] == "step" else 1),
                "flops": 6 * n * dk * dv}
    if case["op"] == "groupnorm":
        n, stats, per = case["N"] * case["S"] * case["C"], 8 * case["N"] * case["G"], 8 * case["C"]
        if case["form"] == "fwd":  # X in, Y and the statistics out
            return {"bytes": 2 * e * n + stats + (per if case["affine"] else 0), "flops": 12 * n}
        return {"bytes": 3 * e * n + stats + (2 * per if case["affine"] else 0), "flops": 24 * n}
    # a block of Philox is 20 products of 32 bits and about 50 other operations for 4 elements
    return {"bytes": case["n"] * e * (3 if case["residual"] else 2), "flops": 18 * case["n"]}


def _exact_delta(case, s):
    B, H, T, dk, dv, lay = (case[k] for k in ("B", "H", "T", "dk", "dv", "layout"))
    if case["form"] == "bwd" and 8 * B * H * (T + 1) * dk * dv > 60e9:
        return None

    def tokens(name, d=None):  # one [B H, d] slice a token
        t = s[name].double()
        t = t.permute(1, 0, 2, 3) if lay == "bthd" and d else t.permute(2, 0, 1, 3) if d else \
            t.permute(1, 0, 2) if lay == "bthd" else t.permute(2, 0, 1)
        if t.shape[2] != H:
            t = t.repeat_interleave(H // t.shape[2], 2)
        return t.reshape(T, B * H, d) if d else t.reshape(T, B * H)

    def back(t):               # and from [T, B H, ...] to the case's layout
        t = t.view(T, B, H, *t.shape[2:])
        t = t.transpose(0, 1) if lay == "bthd" else t.movedim(0, 2)
        return t.contiguous()

    K, Q, V, eta, g = tokens("K", dk), tokens("Q", dk), tokens("V", dv), tokens("eta"), tokens("g")
    a = torch.exp(g)
    zero = torch.zeros(B * H, dv, dk, dtype=torch.float64, device=K.device)
    W = zero if s["W"] is None else s["W"].double().reshape(B * H, dv, dk)
    bwd = case["form"] == "bwd"
    Z = None if bwd else torch.empty_like(V)
    before = torch.empty(T, B * H, dv, dk, dtype=torch.float64, device=K.device) if bwd else None
    err = torch.empty_like(V) if bwd else None
    for t in range(T):
        k = K[t][:, None]
        if bwd:
            before[t] = W
        W = W * a[t][:, None, None]
        u = V[t] - (W * k).sum(2)
        W = W + (u * eta[t][:, None])[:, :, None] * k
        if bwd:
            err[t] = u
        else:
            Z[t] = (W * Q[t][:, None]).sum(2)
    if not bwd:
        return back(Z), W.view(B, H, dv, dk)
    dZ = tokens("dZ", dv)
    D = zero if s["dW"] is None else s["dW"].double().reshape(B * H, dv, dk)
    dK, dQ, dV, deta, dg = (torch.empty_like(t) for t in (K, Q, V, eta, g))
    for t in range(T - 1, -1, -1):
        k, u = K[t][:, None], err[t]
        D = D + dZ[t][:, :, None] * Q[t][:, None]
        kept = before[t] * a[t][:, None, None]
        now = kept + (u * eta[t][:, None])[:, :, None] * k
        dQ[t] = (now * dZ[t][:, :, None]).sum(1)
        du = (D * k).sum(2)
        deta[t] = (du * u).sum(1)
        dV[t] = du * eta[t][:, None]
        dK[t] = (D * (u * eta[t][:, None])[:, :, None]).sum(1) - (kept * dV[t][:, :, None]).sum(1)
        D = D - dV[t][:, :, None] * k
        dg[t] = (D * kept).sum((1, 2))
        D = D * a[t][:, None, None]
    dK, dQ = ((t.view(T, B, -1, case["share"], dk).sum(3)) for t in (dK, dQ))
    keys = [t.transpose(0, 1).contiguous() if lay == "bthd" else t.movedim(0, 2).contiguous() for t in (dK, dQ)]
    return keys[0], keys[1], back(dV), back(deta), back(dg), D.view(B, H, dv, dk)


def _exact_groupnorm(case, s):
    N, S, C, G = (case[k] for k in "NSCG")
    per = C // G
    x = s["X"].double().view(N, S, G, per).permute(0, 2, 1, 3).reshape(N, G, S * per)
    ones = torch.ones(C, dtype=torch.float64, device=x.device)
    w = ones if s["w"] is None else s["w"].double()
    b = 0.0 * ones if s["b"] is None else s["b"].double()
    wide = [t.view(G, 1, per).expand(G, S, per).reshape(G, S * per) for t in (w, b)]

    def back(t):
        return t.view(N, G, S, per).permute(0, 2, 1, 3).reshape(N, S, C)

    if case["form"] == "fwd":
        var, mean = torch.var_mean(x, 2, correction=0)
        rstd = (var + _EPS) ** -0.5
    else:
        mean, rstd = s["mean"].double(), s["rstd"].double()
    n = (x - mean[..., None]) * rstd[..., None]
    v = n * wide[0] + wide[1]
    normal = torch.distributions.Normal(torch.zeros((), dtype=torch.float64, device=x.device), 1.0)
    if case["form"] == "fwd":
        y = v / (1.0 + torch.exp(-v)) if case["act"] == "silu" else v * normal.cdf(v) if case["act"] == "gelu" else v
        return back(y), mean, rstd
    dy = s["dY"].double().view(N, S, G, per).permute(0, 2, 1, 3).reshape(N, G, S * per)
    if case["act"] == "silu":
        dy = dy * (1.0 + torch.exp(-v) * (1.0 + v)) / (1.0 + torch.exp(-v)) ** 2
    elif case["act"] == "gelu":
        dy = dy * (normal.cdf(v) + v * torch.exp(normal.log_prob(v)))
    dn = dy * wide[0]
    m = S * per
    dx = (dn - dn.sum(2, keepdim=True) / m - n * ((dn * n).sum(2, keepdim=True) / m)) * rstd[..., None]
    if not case["affine"]:
        return back(dx), None, None
    return back(dx), back(dy * n).sum((0, 1)), back(dy).sum((0, 1))


def _exact_dropout(case, s):
    n, (seed, first) = case["n"], (int(v) for v in s["rng"].tolist())
    word, mask, half = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    at = np.arange((n + 3) // 4, dtype=word) + word(first % (1 << 64))
    x = [at & mask, at >> half, np.zeros_like(at), np.zeros_like(at)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for r in range(10):
        p, q = x[0] * word(0xD2511F53), x[2] * word(0xCD9E8D57)
        k = [word((key[0] + r * 0x9E3779B9) % (1 << 32)), word((key[1] + r * 0xBB67AE85) % (1 << 32))]
        x = [(q >> half) ^ x[1] ^ k[0], q & mask, (p >> half) ^ x[3] ^ k[1], p & mask]
    keep = np.stack(x, 1).reshape(-1)[:n].astype(np.float64) / 4294967296.0 >= case["p"]
    keep = torch.from_numpy(keep).to(s["X"].device)
    y = torch.where(keep, s["X"].double() / (1.0 - case["p"]), 0.0)
    return y if s["res"] is None else y + s["res"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "delta":
        return _exact_delta(case, s)
    return _exact_groupnorm(case, s) if case["op"] == "groupnorm" else _exact_dropout(case, s)
