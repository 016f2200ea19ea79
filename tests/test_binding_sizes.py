"""Sizes beyond 32 bits are refused by the binding, before the library would see their lower bits (no GPU
needed: the tensors are shapes alone)."""
import pytest

from test_sequence_layers_ttt_amd import ttt

BIG = (1 << 32) + 8


def shape(*s, dt=None):
    import torch
    return torch.empty(s, dtype=dt or torch.bfloat16, device="meta")


def beyond():
    return pytest.raises(ValueError, match="beyond the library's 32 bits")


@pytest.mark.parametrize("s", [(1, 1, BIG, 1), (BIG, 1, 1, 1), (1, BIG, 1, 8), (1, 1, 4, BIG)])
def test_recurrence(s):
    import torch
    X = shape(*s)
    with beyond():
        ttt.gated_fwd(X, X)
    with beyond():
        ttt.gated_step(X, X, shape(s[0], s[1], s[3], dt=torch.float32))
    with beyond():
        ttt.gated_bwd(X, X, X)
    with beyond():
        ttt.gated_workspace_bytes(*s, ttt.DTYPE_BF16)


def test_norm():
    X = shape(1, (1 << 32) + 64)
    for call in (ttt.rmsnorm_fwd, ttt.rmsnorm_q8_fwd, lambda x: ttt.rmsnorm_bwd(x, None, x)):
        with beyond():
            call(X)
    with beyond():
        ttt.rmsnorm_bwd_workspace_bytes(1, (1 << 32) + 64, ttt.DTYPE_BF16)
    # as many rows as there are: their number is 64 bits wide
    with pytest.raises(ValueError, match="device tensor"):
        ttt.rmsnorm_fwd(shape(BIG, 64))
    assert ttt.rmsnorm_bwd_workspace_bytes(BIG, 64, ttt.DTYPE_BF16) > 0


def test_scan():
    X, W = shape(1, 1, BIG, 4), shape(1, 1, 4, 4)
    for call in (lambda: ttt.linear_fwd(X, X, X, None, W, 16), lambda: ttt.linear_bwd(X, X, X, None, W, X, 16),
                 lambda: ttt.linear_fwd_noalloc(X, X, X, None, W, 16, Z=X, W_out=W),
                 lambda: ttt.linear_step(X, X, X, None, W, W, 0, 16),
                 lambda: ttt.linear_fwd_momentum(X, X, X, None, W, None, 0.9, 16),
                 lambda: ttt.linear_ln_fwd(X, X, X, None, W, X, None, None, 16),
                 lambda: ttt.mlp_fwd(X, X, X, None, W, None, W, None, 16),
                 lambda: ttt.linear_fwd_varlen(X[0], X[0], X[0], None, W, shape(2), 16)):
        with beyond():
            call()
    for query in (ttt.linear_workspace_bytes, ttt.mlp_workspace_bytes):
        with beyond():
            query(1, 1, BIG, 64, 16)
        with beyond():
            query(1, 1, 64, 64, (1 << 32) + 16)
    for query in (ttt.linear_select_plan, ttt.mlp_select_plan, ttt.linear_bwd_workspace_bytes,
                  ttt.linear_select_plan_varlen):
        with beyond():
            query(1, 1, 64, 64, (1 << 32) + 16, ttt.DTYPE_BF16)
        with beyond():
            query(1, 1, -(1 << 32) + 64, 64, 16, ttt.DTYPE_BF16)
