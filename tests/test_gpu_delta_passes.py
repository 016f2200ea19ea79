"""The gated delta rule where a call takes its heads in several passes, past 2^31 elements backward, and
with wide fp32 heads that share keys."""
import pytest

import delta_ref as ref
from gpu_helpers import say
from test_gpu_delta import Case, check_bwd, check_fwd
from test_gpu_delta_block import tensors
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def alone(c, b, h):
    """The tensors of one batch and the head h of keys with the heads of values that share it."""
    s = slice(b, b + 1)
    keys = [t[s, :, h:h + 1] for t in (c.K, c.Q)]
    values = [t[s, :, h * c.share:(h + 1) * c.share] for t in (c.V, c.eta, c.g)]
    states = [t[s, h * c.share:(h + 1) * c.share] for t in (c.W0, c.dW)]
    dZ = c.dZ[s, :, h * c.share:(h + 1) * c.share]
    return [t.contiguous() for t in keys + values + states[:1] + [dZ] + states[1:]]


def near_alone(c, got, want, b, h, what):
    """A head out of many against its own call (whose chunks may be cut elsewhere)."""
    rel = 2 * ref.delta_rel(c.T, c.dk, c.dv)
    for i, (x, y) in enumerate(zip(got, want)):
        x = x[b:b + 1, h * y.shape[1]:(h + 1) * y.shape[1]] if what[i] == "state" else \
            x[b:b + 1, :, h * y.shape[2]:(h + 1) * y.shape[2]]
        assert x.shape == y.shape, i
        half = 2 * ref.HALF[c.io] + (2 * ref.Z_BF16 if c.io == "bf16" else 0) if what[i] == "tokens" else 0.0
        err = (x.double() - y.double()).abs().max().item()
        # (dg's parts cancel: about ten times its largest value goes into the sum)
        assert err <= (rel * (10 if what[i] == "dg" else 1) + half) * y.double().abs().max().item(), (b, h, i, err)


@pytest.mark.parametrize("shape", [(43, 16, 1, 5200, 16, 16), (22, 32, 2, 5184, 16, 20)])
def test_forward_in_passes(dev, shape):
    """Past a gigabyte of workspace; the last pass has fewer heads than the others."""
    B, H, share, T, dk, dv = shape
    c = Case(dev, *shape, "bf16", ttt.LAYOUT_BTHD, seed=sum(shape))
    # 21.5 KB a chunk: more chunks of heads than one pass of 2^30 bytes has, and its bytes stay below
    units = B * H * ((T + 63) // 64)
    need = ttt.delta_workspace_bytes(B, H, H // share, T, dk, dv, 1)
    assert need <= 1 << 30 < units * 21500
    got = ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, layout=c.layout)
    for b, h in ((0, 0), (B // 2, 3), (B - 2, H // share - 1), (B - 1, 0), (B - 1, H // share - 1)):
        p = alone(c, b, h)
        near_alone(c, got, ttt.delta_fwd(*p[:6], layout=c.layout), b, h, ("tokens", "state"))


@pytest.mark.parametrize("shape", [(43, 16, 1, 5200, 16, 16), (22, 32, 2, 5184, 16, 20)])
def test_backward_in_passes(dev, shape):
    """Past four gigabytes."""
    B, H, share, T, dk, dv = shape
    c = Case(dev, *shape, "bf16", ttt.LAYOUT_BTHD, seed=sum(shape))
    units = B * H * ((T + 63) // 64)
    need = ttt.delta_bwd_workspace_bytes(B, H, H // share, T, dk, dv, 1)
    assert need <= 4 << 30 < units * 81000
    got = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW, layout=c.layout)
    for b, h in ((0, 0), (B // 2, 3), (B - 2, H // share - 1), (B - 1, 0), (B - 1, H // share - 1)):
        want = ttt.delta_bwd(*alone(c, b, h), layout=c.layout)
        near_alone(c, got, want, b, h, ("tokens", "tokens", "tokens", "gates", "dg", "state"))


def test_backward_past_32_bits(dev):
    """More than 2^31 elements of keys in one head: the gradients of a document that starts anew near
    the end are what they are alone, and the others get none."""
    import torch
    T, d, dv, n = (1 << 24) + 64 + 40, 128, 16, 104
    K = torch.zeros(1, 1, T, d, dtype=torch.bfloat16, device=dev)
    V, dZ = (torch.zeros(1, 1, T, dv, dtype=torch.bfloat16, device=dev) for _ in range(2))
    eta, g = torch.full((1, 1, T), 0.5, device=dev), torch.zeros(1, 1, T, device=dev)
    k, = tensors(dev, 52, (1, 1, n, d))
    K[:, :, -n:] = torch.nn.functional.normalize(k, dim=-1).bfloat16()
    V[:, :, -n:], dZ[:, :, -n:] = tensors(dev, 53, *[(1, 1, n, dv)] * 2, dt=torch.bfloat16)
    g[:, :, -n] = -float("inf")
    say("bytes of workspace", ttt.delta_bwd_workspace_bytes(1, 1, 1, T, d, dv, 1))
    got = ttt.delta_bwd(K, K, V, eta, g, None, dZ)
    tail = [t[:, :, -n:].clone() for t in (K, K, V, eta, g)]
    want = ttt.delta_bwd(*tail, None, dZ[:, :, -n:].clone())
    rel = 2 * ref.delta_rel(n, d, dv)
    for i, (a, b) in enumerate(zip(got[:5], want)):
        # (chunks end elsewhere: two roundings to bf16 of nearly the same values)
        more = 2 * ref.HALF["bf16"] if i < 3 else 10 * rel
        assert (a[:, :, -n:].double() - b.double()).abs().max() <= (rel + more) * b.double().abs().max(), i
        assert (a[:, :, :-n] == 0).all(), i
    assert (got[5] == 0).all()


@pytest.mark.parametrize("shape", [(3, 32, 2, 130, 128, 128), (2, 32, 4, 100, 128, 128), (10, 16, 2, 70, 128, 256),
                                   (10, 32, 4, 65, 100, 64), (1, 8, 4, 1700, 128, 128)])
def test_wide_fp32_heads_that_share_keys(dev, shape):
    c = Case(dev, *shape, "f32", seed=sum(shape))
    check_fwd(c, *ttt.delta_fwd(c.K, c.Q, c.V, c.eta, c.g, c.W0))
    got = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    check_bwd(c, got)
    again = ttt.delta_bwd(c.K, c.Q, c.V, c.eta, c.g, c.W0, c.dZ, c.dW)
    assert all((x == y).all() for x, y in zip(got, again))
