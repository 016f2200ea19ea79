"""Inputs of a long memory for the gated recurrence, with an error bound that does not grow with the
memory.

The kernels compose affine maps.  A token's value passes on its way to an output through at most

    8 tokens, 16 runs, 16 parts, 7 tiles and 1 group          (the pairs it becomes part of)
    NG groups                                                 (the chain of the groups' states)
    1 tile, 16 parts, 1 run and 8 tokens                      (from the group's state to the output)

compositions fma(exp2(S), h, B), 74 + NG together.  In each the exponential is off by 2 half-steps and the
sum by 1; S is a sum of up to 48 roundings' worth, each product g log2(e) off by 1.5, so that it is off by at
most 50 |S| half-steps, and |S| exp(S) <= 0.37: 18.5.  That makes 22 half-steps of the values composed, and
those are no larger than twice the largest |z| of the channel, since a map's B is the difference of a state
and a decayed state.  The factors are at most 1: errors are carried on and never grow."""
import numpy as np

U = 2.0 ** -24


def bound(z, groups):
    """Of every value of z [N, T, d] (or of a row's last), before the output's rounding."""
    with np.errstate(invalid="ignore"):
        big = np.abs(z).max(1, keepdims=True)
    return 22 * (74 + groups) * U * 2 * big


def gates(kind, gen, *shape):
    """Gates of a long memory, fp64."""
    if kind == "carry":
        return np.zeros(shape)
    if kind == "slow":
        return np.full(shape, -1e-4)
    # a trained layer's, of a memory of some 10^4 tokens
    return -np.log1p(np.exp(-(gen.standard_normal(shape) + 9.5)))


def drifting(gen, N, T, d, every):
    """x whose mean changes from stretch to stretch, so that no tile's share is like another's."""
    mean = np.repeat(gen.standard_normal((N, -(-T // every), d)), every, 1)[:, :T]
    return 0.3 * gen.standard_normal((N, T, d)) + 0.1 * mean
