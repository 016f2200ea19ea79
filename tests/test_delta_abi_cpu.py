"""Host-side refusals of the gated delta rule, group norm and dropout: every call here carries an
argument that the validation refuses, so nothing is launched (no GPU needed)."""
import math

import pytest

from test_sequence_layers_ttt_amd import ttt

P = [0x10000000 * (k + 1) for k in range(20)]     # far apart, aligned, never dereferenced
BIG = 1 << 40


def delta(**kw):
    a = dict(K=P[0], Q=P[1], V=P[2], eta=P[3], es=0.0, g=P[4], W0=P[5], Z=P[6], W=P[7], B=2, H=4, Hk=2, T=100,
             dk=64, dv=64, lay=0, io=1, ws=P[8], wsb=BIG)
    a.update(kw)
    return ttt.lib().ttt_delta_fwd(*(a[k] for k in ("K", "Q", "V", "eta", "es", "g", "W0", "Z", "W", "B", "H", "Hk",
                                                    "T", "dk", "dv", "lay", "io", "ws", "wsb")), None)


BAD_DELTA = [
    dict(K=None), dict(Q=None), dict(V=None), dict(K=P[0] + 8), dict(Q=P[1] + 2), dict(V=P[2] + 4),
    dict(W0=P[5] + 4), dict(eta=P[3] + 2), dict(g=P[4] + 1), dict(B=0), dict(H=0), dict(Hk=0), dict(Hk=3),
    dict(T=0), dict(dk=0), dict(dv=-1), dict(lay=2), dict(lay=-1), dict(io=2), dict(T=(1 << 30) + 1),
    dict(eta=None, es=math.nan), dict(eta=None, es=math.inf), dict(B=1 << 20, H=1 << 10, Hk=1),
    dict(B=1 << 10, H=1 << 10, Hk=1, T=1 << 28), dict(B=1 << 22, H=1, Hk=1), dict(B=1, H=4, Hk=1, T=1 << 28),
]


@pytest.mark.parametrize("kw", BAD_DELTA + [
    dict(Z=None), dict(Z=P[6] + 8), dict(W=P[7] + 4), dict(Z=P[0]), dict(Z=P[1] + 16), dict(Z=P[2]), dict(Z=P[3]),
    dict(Z=P[4]), dict(Z=P[5]), dict(W=P[6]), dict(W=P[0]), dict(W=P[5] + 16),
])
def test_delta_fwd_refuses(kw):
    assert delta(**kw) == ttt.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(dk=129), dict(dv=257), dict(dk=1 << 20)])
def test_delta_widths_past_the_kernels_are_unsupported(kw):
    assert delta(**kw) == ttt.ERR_UNSUPPORTED


@pytest.mark.parametrize("T", [17, 64, 65, 4097])
def test_delta_workspace_is_asked_for(T):
    need = ttt.delta_workspace_bytes(2, 4, 2, T, 64, 64, 1)
    assert need > 0
    assert delta(T=T, ws=None) == ttt.ERR_WORKSPACE
    assert delta(T=T, wsb=need - 1) == ttt.ERR_WORKSPACE
    assert delta(T=T, ws=P[8] + 128) == ttt.ERR_WORKSPACE


def step(**kw):
    a = dict(K=P[0], Q=P[1], V=P[2], eta=P[3], es=0.0, g=P[4], W=P[5], Z=P[6], B=2, H=4, Hk=2, T=3, dk=64, dv=64,
             lay=0, io=1)
    a.update({("W" if k == "W0" else k): v for k, v in kw.items()})
    return ttt.lib().ttt_delta_step(*(a[k] for k in ("K", "Q", "V", "eta", "es", "g", "W", "Z", "B", "H", "Hk", "T",
                                                     "dk", "dv", "lay", "io")), None)


@pytest.mark.parametrize("kw", BAD_DELTA + [dict(W=None), dict(Z=None), dict(Z=P[5]), dict(Z=P[2]), dict(W=P[0])])
def test_delta_step_refuses(kw):
    assert step(**kw) == ttt.ERR_INVALID_ARG


def bwd(**kw):
    names = ("K", "Q", "V", "eta", "es", "g", "W0", "dZ", "dWT", "dK", "dQ", "dV", "deta", "dg", "dW0", "B", "H",
             "Hk", "T", "dk", "dv", "lay", "io", "ws", "wsb")
    a = dict(K=P[0], Q=P[1], V=P[2], eta=P[3], es=0.0, g=P[4], W0=P[5], dZ=P[6], dWT=P[7], dK=P[8], dQ=P[9],
             dV=P[10], deta=P[11], dg=P[12], dW0=P[13], B=2, H=4, Hk=2, T=100, dk=64, dv=64, lay=0, io=1, ws=P[14],
             wsb=BIG)
    a.update(kw)
    return ttt.lib().ttt_delta_bwd(*(a[k] for k in names), None)


@pytest.mark.parametrize("kw", BAD_DELTA + [
    dict(dZ=None), dict(dK=None), dict(dQ=None), dict(dV=None), dict(dZ=P[6] + 4), dict(dWT=P[7] + 8),
    dict(dK=P[8] + 2), dict(deta=P[11] + 2), dict(dg=P[12] + 1), dict(dW0=P[13] + 4), dict(dK=P[0]), dict(dQ=P[8]),
    dict(dV=P[6]), dict(dW0=P[5]), dict(dW0=P[7]), dict(deta=P[3]), dict(dg=P[11]),
])
def test_delta_bwd_refuses(kw):
    assert bwd(**kw) == ttt.ERR_INVALID_ARG


@pytest.mark.parametrize("T", [1, 64, 4097])
def test_delta_bwd_workspace_is_asked_for(T):
    need = ttt.delta_bwd_workspace_bytes(2, 4, 2, T, 64, 64, 1)
    assert need > 0
    assert bwd(T=T, ws=None) == ttt.ERR_WORKSPACE
    assert bwd(T=T, wsb=need - 1) == ttt.ERR_WORKSPACE
    assert bwd(T=T, ws=P[14] + 128) == ttt.ERR_WORKSPACE


def group(**kw):
    a = dict(X=P[0], w=P[1], b=P[2], eps=1e-5, act=1, Y=P[3], mean=P[4], rstd=P[5], N=4, S=100, C=64, G=8, io=1,
             ws=P[6], wsb=BIG)
    a.update(kw)
    return ttt.lib().ttt_groupnorm_fwd(*(a[k] for k in ("X", "w", "b", "eps", "act", "Y", "mean", "rstd", "N", "S",
                                                        "C", "G", "io", "ws", "wsb")), None)


BAD_GROUP = [
    dict(X=None), dict(mean=None), dict(rstd=None), dict(X=P[0] + 8), dict(w=P[1] + 2), dict(b=P[2] + 1),
    dict(mean=P[4] + 2), dict(rstd=P[5] + 2), dict(N=-1), dict(S=-1), dict(C=0), dict(G=0), dict(G=7), dict(G=128),
    dict(C=(1 << 20) + 8), dict(io=2), dict(act=3), dict(act=-1), dict(N=1 << 31, S=1), dict(N=1 << 40, S=1 << 20),
]


@pytest.mark.parametrize("kw", BAD_GROUP + [
    dict(Y=None), dict(Y=P[3] + 8), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
    dict(eps=1e-40), dict(Y=P[0] + 16), dict(Y=P[1]), dict(mean=P[5]), dict(mean=P[3]), dict(rstd=P[0]),
])
def test_groupnorm_fwd_refuses(kw):
    assert group(**kw) == ttt.ERR_INVALID_ARG


def test_groupnorm_of_nothing_does_nothing():
    assert group(N=0, X=None) == ttt.OK and group(S=0, Y=None) == ttt.OK


def test_groupnorm_workspace_is_asked_for():
    need = ttt.groupnorm_workspace_bytes(4, 100000, 64, 8, 1)
    assert need > 0
    assert group(S=100000, ws=None) == ttt.ERR_WORKSPACE
    assert group(S=100000, wsb=need - 1) == ttt.ERR_WORKSPACE
    for S in (1, 100):
        assert ttt.groupnorm_workspace_bytes(4, S, 64, 8, 1) == 0


def group_bwd(**kw):
    names = ("X", "w", "b", "act", "mean", "rstd", "dY", "dX", "dw", "db", "N", "S", "C", "G", "io", "ws", "wsb")
    a = dict(X=P[0], w=P[1], b=P[2], act=1, mean=P[3], rstd=P[4], dY=P[5], dX=P[6], dw=P[7], db=P[8], N=4, S=100,
             C=64, G=8, io=1, ws=P[9], wsb=BIG)
    a.update(kw)
    return ttt.lib().ttt_groupnorm_bwd(*(a[k] for k in names), None)


@pytest.mark.parametrize("kw", BAD_GROUP[:3] + [
    dict(dY=None), dict(dX=None), dict(dX=P[6] + 4), dict(dY=P[5] + 2), dict(dw=P[7] + 2), dict(db=P[8] + 2),
    dict(dX=P[0] + 64), dict(dX=P[5] + 64), dict(dX=P[1]), dict(dw=P[1]), dict(dw=P[8]), dict(db=P[0]),
    dict(dw=P[5]), dict(db=P[6]), dict(dX=P[3]), dict(act=5), dict(G=5), dict(N=-2), dict(io=9),
])
def test_groupnorm_bwd_refuses(kw):
    assert group_bwd(**kw) == ttt.ERR_INVALID_ARG


def test_groupnorm_bwd_workspace_is_asked_for():
    for S in (1, 100, 100000):
        need = ttt.groupnorm_bwd_workspace_bytes(4, S, 64, 8, 1)
        assert need > 0
        assert group_bwd(S=S, ws=None) == ttt.ERR_WORKSPACE
        assert group_bwd(S=S, wsb=need - 1) == ttt.ERR_WORKSPACE


def drop(**kw):
    a = dict(X=P[0], R=P[1], Y=P[2], n=1000, p=0.1, rng=P[3], io=1)
    a.update(kw)
    return ttt.lib().ttt_dropout(*(a[k] for k in ("X", "R", "Y", "n", "p", "rng", "io")), None)


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(Y=None), dict(rng=None), dict(X=P[0] + 8), dict(R=P[1] + 2), dict(Y=P[2] + 4),
    dict(rng=P[3] + 4), dict(n=-1), dict(n=1 << 60), dict(p=1.0), dict(p=-0.1), dict(p=math.nan), dict(io=3),
    dict(Y=P[0] + 16), dict(Y=P[1] + 16), dict(Y=P[3]),
])
def test_dropout_refuses(kw):
    assert drop(**kw) == ttt.ERR_INVALID_ARG


def test_dropout_of_nothing_does_nothing():
    assert drop(n=0, X=None) == ttt.OK


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    K, eta = torch.zeros(1, 2, 20, 16), torch.zeros(1, 2, 20)
    with pytest.raises(ValueError):                     # host tensors
        ttt.delta_fwd(K, K, K, eta)
    with pytest.raises(ValueError):
        ttt.delta_step(K, K, K, eta, None, None)        # a step needs its state
    with pytest.raises(ValueError):
        ttt.delta_fwd(K, K, K, eta, layout=2)
    with pytest.raises(ValueError):
        ttt.delta_fwd(K[0], K[0], K[0], eta)
    with pytest.raises(ValueError):
        ttt.groupnorm_fwd(K, 3)
    with pytest.raises(ValueError):
        ttt.groupnorm_fwd(K, 4)
    with pytest.raises(ValueError):
        ttt.dropout(K, 0.1, torch.zeros(2, dtype=torch.int64))
