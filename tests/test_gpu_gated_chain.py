"""The recurrence over many groups of tiles with a memory that outlasts them: what enters a group is still
there at its end, so every link of the chain shows in the results.  Forward, backward, and with the state in
place, within a bound that a mistake in the chain is far outside of (test_gated_chain.py)."""
import numpy as np
import pytest

import block_ref as ref
import chain_ref as chain
from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


# (rows, tokens, tokens of a group, features, type): more than nine groups each
SHAPES = [(3, 40000, 2048, 64, "bf16"), (2, 40000, 2048, 64, "f32"), (3, 12007, 768, 83, "f32"),
          (2, 11000, 704, 520, "bf16"), (2, 90001, 8192, 16, "bf16"), (1, 20479, 1024, 200, "f32")]


def np64(t):
    return t.double().cpu().numpy()[0]


@pytest.mark.parametrize("resets", [False, True])
@pytest.mark.parametrize("kind", ["slow", "trained", "carry"])
@pytest.mark.parametrize("N,T,per,d,io", SHAPES)
def test_long_memory(dev, N, T, per, d, io, kind, resets):
    import torch
    say("case", N, T, d, io, kind, resets)
    gen = np.random.default_rng(T + d)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    on = lambda a, t=dt: torch.from_numpy(a.astype(np.float32))[None].to(dev, t)  # noqa: E731
    g = chain.gates(kind, gen, N, T, d)
    if resets:      # of some channels alone, in a group in the middle and in one near the end
        g[:, 4 * per + per // 3, ::3] = -np.inf
        g[:, (T // per - 1) * per - 5, 1::4] = -np.inf
    G, X, dZ = on(g), on(chain.drifting(gen, N, T, d, per // 8)), on(chain.drifting(gen, N, T, d, per // 8))
    h0, dh = (on(5 * gen.standard_normal((N, d)), torch.float32) for _ in range(2))
    groups = -(-T // per)

    Z, hT = ttt.gated_fwd(X, G, h0)
    want = ref.gated(np64(X), np64(G), np64(h0))
    room = chain.bound(want, groups)
    ok, worst = ref.within(np64(Z), want, room, io)
    ok2, worst2 = ref.within(np64(hT), want[:, -1], room[:, 0], "f32")
    say("  error over what is allowed: Z %.3f h_T %.3f" % (worst, worst2))
    assert ok and ok2
    h = h0.clone()
    Z2, _ = ttt.gated_fwd(X, G, h, h_out=h)
    assert torch.equal(Z, Z2) and torch.equal(hT, h)

    got = ttt.gated_bwd(G, Z, dZ, h0, dh)
    a, z = np64(G), np64(Z)
    shut = np.isneginf(a)
    lam, dG, dh0 = ref.gated_bwd(a, z, np64(h0), np64(dZ), np64(dh))
    room = chain.bound(lam, groups)
    before = np.abs(np.concatenate([np64(h0)[:, None], z[:, :-1]], 1))
    own = (6 + 3 * np.where(shut, 0.0, np.abs(a))) * ref.U       # the gate, its exponential, two products
    for name, x, y, allowed, kind_of in (("dX", got[0], lam, room, io),
                                         ("dG", got[1], dG, np.where(shut, 0.0, room * before + own * np.abs(dG)), io),
                                         ("dh0", got[2], dh0, (room + own * np.abs(dh0)[:, None])[:, 0], "f32")):
        ok, worst = ref.within(np64(x), y, allowed, kind_of)
        say("  error over what is allowed: %s %.3f" % (name, worst))
        assert ok, name
