"""The recurrence's state in place (h_out at h0) over rows of several groups of tiles with resets in them:
a group with a reset in it hands its state on without waiting for the tiles that read h0, so the row's last
tile has to wait for those itself before it writes there."""
import pytest

from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


# (rows, tokens of a group of 8 tiles, features, type); a tile is 8 tokens of 256 threads over the row's
# 16-byte vectors, or over one line of them where rows are whole lines
SHAPES = [(48, 2048, 64, "bf16"), (5, 2048, 64, "f32"), (20, 768, 83, "f32"), (3, 2048, 520, "bf16"),
          (200, 8192, 16, "bf16"), (1, 16384, 1, "f32")]


@pytest.mark.parametrize("groups", [(1,), (2,), (3,), (1, 2, 3), (4,)])
@pytest.mark.parametrize("N,per,d,io", SHAPES)
def test_resets_in_later_groups(dev, N, per, d, io, groups):
    import torch
    T = 5 * per + 77
    say("case", N, T, d, io, groups)
    gen = torch.Generator(device="cpu").manual_seed(N + d)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    X = torch.randn(1, N, T, d, generator=gen).to(dev, dt)
    # gates of a long memory: what enters the first tile is still there at the end of the row's first group
    G = (-0.01 * torch.rand(1, N, T, d, generator=gen)).to(dev, dt)
    h0 = torch.randn(1, N, d, generator=gen).to(dev) * 100
    for g in groups:
        G[:, :, g * per + per // 3 + 5] = -float("inf")
    Z, hT = ttt.gated_fwd(X, G, h0)
    noise, side = torch.zeros(1 << 22, device=dev), torch.cuda.Stream()
    for k in range(6):
        h = h0.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):      # other work on the card, so that workgroups start unevenly
            for _ in range(k):
                noise.add_(1.0)
        Z2, _ = ttt.gated_fwd(X, G, h, h_out=h)
        torch.cuda.synchronize()
        assert torch.equal(Z, Z2) and torch.equal(hT, h)
