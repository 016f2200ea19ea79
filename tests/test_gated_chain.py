"""What the tests of the recurrence over many groups of tiles would notice: a chain with a mistake planted in
it, in fp64 on the CPU, against the bound that the kernels are held to."""
import numpy as np
import pytest

import block_ref as ref
import chain_ref as chain

GROUP, TILE = 2048, 256


def states(g, x, h0, mistake=None):
    """The states by tiles and groups as the kernels form them, with a mistake in the chain."""
    T, d = x.shape
    z = np.empty_like(x)

    def pair(a, b):
        """(sum of g, state from 0) of tokens a to b"""
        h = np.zeros(d)
        for t in range(a, b):
            h = np.exp(g[t]) * h + x[t]
        return g[a:b].sum(0), h

    enters, before = [np.zeros(d) + h0], None          # the state that enters each group; the last group's pair
    for a in range(0, T, GROUP):
        b, h = min(a + GROUP, T), enters[-1]
        tiles = [pair(t, min(t + TILE, b)) for t in range(a, b, TILE)]
        for j, t0 in enumerate(range(a, b, TILE)):
            s, p = np.zeros(d), np.zeros(d)
            for k in range(j):
                if mistake == "tile left out" and k == 2:
                    continue
                s, p = s + tiles[k][0], np.exp(tiles[k][0]) * p + tiles[k][1]
            now = np.exp(s) * h + p
            for t in range(t0, min(t0 + TILE, b)):
                now = np.exp(g[t]) * now + x[t]
                z[t] = now
        s, p = np.zeros(d), np.zeros(d)
        for S, B in tiles:
            s, p = s + S, np.exp(S) * p + B
        if mistake == "the pair before alone":
            enters.append(p)
        elif mistake == "a group left out" and a == 3 * GROUP:
            enters.append(h)
        elif mistake == "the pairs in the wrong order" and before is not None:
            enters.append(np.exp(before[0]) * (np.exp(s) * enters[-2] + p) + before[1])
        elif mistake == "the sum of one tile":
            enters.append(np.exp(tiles[0][0]) * h + p)
        else:
            enters.append(np.exp(s) * h + p)
        before = (s, p)
    return z


MISTAKES = ["the pair before alone", "a group left out", "the pairs in the wrong order", "the sum of one tile",
            "tile left out"]


@pytest.mark.parametrize("kind", ["slow", "trained", "carry"])
def test_mistakes_in_the_chain_are_seen(kind):
    gen = np.random.default_rng(3)
    T, d = 11 * GROUP + 300, 4
    g, x = chain.gates(kind, gen, T, d), chain.drifting(gen, 1, T, d, TILE)[0]
    h0 = 5 * gen.standard_normal(d)
    want = ref.gated(x[None], g[None], h0[None])
    room = chain.bound(want, 12)
    assert ref.within(states(g, x, h0)[None], want, room, "f32")[1] < 1e-3
    for mistake in MISTAKES:
        if kind == "carry" and mistake in ("the sum of one tile", "the pairs in the wrong order"):
            continue                                   # (with gates of 1 they are none)
        for io in ("f32", "bf16"):
            ok, worst = ref.within(states(g, x, h0, mistake)[None], want, room, io)
            assert not ok and worst > 4, (mistake, worst)
