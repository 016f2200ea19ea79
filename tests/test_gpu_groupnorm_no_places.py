"""Rows without places have no statistics, and no memory of before in their place."""
import pytest

from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(3, 0, 32), (5, 4, 0, 32)])
def test_statistics_of_no_places(shape):
    import torch
    dev = torch.device("cuda:0")
    torch.ones(shape[0], 4, device=dev)          # (what the allocator would hand out again)
    w = torch.ones(32, device=dev)
    X = torch.empty(shape, device=dev)
    Y, mean, rstd = ttt.groupnorm_fwd(X, 4, w, w)
    assert Y.shape == X.shape and mean.shape == (shape[0], 4)
    assert mean.isnan().all() and rstd.isnan().all()
    given = torch.ones(shape[0], 4, device=dev)
    assert ttt.groupnorm_fwd(X, 4, w, w, mean=given)[1] is given and given.isnan().all()
    dX, dw, db = ttt.groupnorm_bwd(X, 4, w, w, X, mean, rstd)
    assert dX.shape == X.shape and (dw == 0).all() and (db == 0).all()
