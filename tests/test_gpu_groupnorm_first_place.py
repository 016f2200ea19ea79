"""The group norm of large groups whose first place is far from all others, as a sequence's first
token can be."""
import numpy as np
import pytest

import delta_ref as ref
from gpu_helpers import say
from test_gpu_groupnorm import EPS, np64
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


# N, S, C, G, io: a thread takes 16, 170, 512 and 512 places of a channel
SHAPES = [(8, 4096, 640, 32, "bf16"), (300, 1024, 680, 4, "f32"), (512, 1024, 2048, 32, "bf16"),
          (512, 1024, 1024, 32, "f32")]


@pytest.mark.parametrize("far", [300.0, 1000.0, 1e4])
@pytest.mark.parametrize("shape", SHAPES)
def test_statistics(dev, shape, far):
    """rstd to 256 U.  A run of 17 values, the first at a distance D from the others, has sums of 16
    roundings each, so its squares are good to 17^2 U of D^2, half of that in rstd (145 U); in the next
    run the distance to the mean is D / 17, which with those after it adds less than 17 U; joins and
    the reciprocal root are below 40 U."""
    import torch
    N, S, C, G, io = shape
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    assert ttt.groupnorm_workspace_bytes(N, S, C, G, ttt.DTYPE_BF16 if io == "bf16" else ttt.DTYPE_F32) > 0
    gen = torch.Generator(device=dev).manual_seed(S + C)
    X = (0.1 * torch.empty(N, S, C, dtype=dt, device=dev).normal_(generator=gen))
    X[:, 0] += far
    _, mean, rstd = ttt.groupnorm_fwd(X, G, eps=EPS)
    rows = [0, N // 2, N - 1]
    x = ref.groups(np64(X[rows]), G)
    m = x.mean(2)
    r = 1 / np.sqrt(((x - m[..., None]) ** 2).mean(2) + EPS)
    err = np.abs(np64(rstd[rows]) / r - 1).max()
    off = np.abs(np64(mean[rows]) - m).max()
    say("rstd %.1f U, mean %.2g" % (err / ref.U, off))
    assert err <= 256 * ref.U
    # means: 16 roundings of a run's sums and as many of its mean's steps, of at most `far`
    assert (np.abs(np64(mean[rows]) - m) <= 64 * ref.U * far).all()
