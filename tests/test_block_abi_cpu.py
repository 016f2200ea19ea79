"""Host-side refusals of the operators around the scan: every call here carries an argument that
the validation refuses, so nothing is launched (no GPU needed)."""
import ctypes
import math

import pytest

from test_sequence_layers_ttt_amd import ttt

A = 0x10000000            # far apart, aligned, never dereferenced
STEP = 0x10000000
P = [A + k * STEP for k in range(12)]
BIG = 1 << 40


def gated(**kw):
    a = dict(X=P[0], G=P[1], h0=P[2], Z=P[3], h_out=P[4], B=2, H=3, T=40, d=64, io=1, ws=P[5], wsb=BIG)
    a.update(kw)
    return ttt.lib().ttt_gated_fwd(a["X"], a["G"], a["h0"], a["Z"], a["h_out"], a["B"], a["H"],
                                   a["T"], a["d"], a["io"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(G=None), dict(Z=None), dict(X=P[0] + 8), dict(G=P[1] + 2), dict(Z=P[3] + 4),
    dict(h0=P[2] + 4), dict(h_out=P[4] + 8), dict(B=0), dict(H=-1), dict(T=0), dict(d=0),
    dict(io=2), dict(io=-1), dict(B=1 << 20, H=1 << 20), dict(T=1 << 30, d=1 << 30),
    dict(T=(1 << 30) + 1), dict(T=0x7fffffff), dict(d=(1 << 28) + 1), dict(d=0x7fffffff),
    dict(d=(1 << 26) + 1), dict(T=1 << 20, d=(1 << 14) + 1),
    dict(Z=P[0]), dict(Z=P[1] + 16), dict(Z=P[2]), dict(h_out=P[0]), dict(h_out=P[3]),
    dict(h_out=P[2] + 16),                              # a shifted overlap of the states
])
def test_gated_fwd_refuses(kw):
    assert gated(**kw) == ttt.ERR_INVALID_ARG


def bwd(**kw):
    a = dict(G=P[0], Z=P[1], h0=P[2], dZ=P[3], dhT=P[4], dX=P[5], dG=P[6], dh0=P[7], B=2, H=3, T=40,
             d=64, io=0, ws=P[8], wsb=BIG)
    a.update(kw)
    return ttt.lib().ttt_gated_bwd(a["G"], a["Z"], a["h0"], a["dZ"], a["dhT"], a["dX"], a["dG"],
                                   a["dh0"], a["B"], a["H"], a["T"], a["d"], a["io"], a["ws"],
                                   a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(G=None), dict(Z=None), dict(dZ=None), dict(dX=None), dict(dG=None), dict(dZ=P[3] + 4),
    dict(dh0=P[7] + 4), dict(dhT=P[4] + 4), dict(T=-1), dict(io=7), dict(dX=P[3]), dict(dG=P[0]),
    dict(dG=P[5]), dict(dh0=P[2]), dict(dh0=P[4]), dict(dh0=P[5] + 64),
])
def test_gated_bwd_refuses(kw):
    assert bwd(**kw) == ttt.ERR_INVALID_ARG


@pytest.mark.parametrize("T", [1, 64, 257, 4097, 32768])
def test_gated_workspace_is_asked_for(T):
    need = ttt.gated_workspace_bytes(2, 3, T, 64, 1)
    if need:
        assert gated(T=T, ws=None) == ttt.ERR_WORKSPACE
        assert gated(T=T, wsb=need - 1) == ttt.ERR_WORKSPACE
        assert gated(T=T, ws=P[5] + 128) == ttt.ERR_WORKSPACE
        assert bwd(T=T, io=1, ws=None) == ttt.ERR_WORKSPACE
        assert bwd(T=T, io=1, wsb=need - 1) == ttt.ERR_WORKSPACE
    assert ttt.gated_workspace_bytes(0, 3, T, 64, 1) == 0
    assert ttt.gated_workspace_bytes(2, 3, T, 64, 5) == 0


@pytest.mark.parametrize("kw", [dict(X=None), dict(G=None), dict(h=None), dict(Z=None), dict(n=0),
                                dict(h=P[2] + 4), dict(io=3), dict(Z=P[0]), dict(h=P[3])])
def test_gated_step_refuses(kw):
    a = dict(X=P[0], G=P[1], h=P[2], Z=P[3], n=1, io=1)
    a.update(kw)
    assert ttt.lib().ttt_gated_step(a["X"], a["G"], a["h"], a["Z"], 2, 3, a["n"], 64, a["io"],
                                    None) == ttt.ERR_INVALID_ARG


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw", [
    dict(X=None), dict(Y=None), dict(X=P[0] + 8), dict(res=P[1] + 4), dict(w=P[2] + 2),
    dict(Y=P[3] + 8), dict(R=P[5] + 4), dict(rows=-1), dict(D=0), dict(D=-4), dict(io=2),
    dict(D=(1 << 26) + 1), dict(D=(1 << 28) + 1), dict(D=0x7fffffff), dict(eps=0.0), dict(eps=1e-40), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(rows=1 << 62),
    dict(Y=P[1]), dict(Y=P[0] + 16), dict(R=P[3]), dict(R=P[0] + 32), dict(R=P[1] + 16), dict(w=P[3]),
    dict(w=P[5]),
])
def test_rmsnorm_fwd_refuses(kw, q8):
    a = dict(X=P[0], res=P[1], w=P[2], eps=1e-6, Y=P[3], scale=P[4], R=P[5], rows=9, D=64, io=1)
    a.update(kw)
    L = ttt.lib()
    if q8:
        rc = L.ttt_rmsnorm_q8_fwd(a["X"], a["res"], a["w"], a["eps"], a["Y"], a["scale"], a["R"],
                                  a["rows"], a["D"], a["io"], None)
    else:
        rc = L.ttt_rmsnorm_fwd(a["X"], a["res"], a["w"], a["eps"], a["Y"], a["R"], a["rows"], a["D"],
                               a["io"], None)
    assert rc == ttt.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(scale=None), dict(scale=P[4] + 2), dict(scale=P[0]),
                                dict(scale=P[3]), dict(scale=P[5]), dict(Y=P[0])])
def test_rmsnorm_q8_refuses(kw):
    a = dict(Y=P[3], scale=P[4])
    a.update(kw)
    assert ttt.lib().ttt_rmsnorm_q8_fwd(P[0], P[1], P[2], 1e-6, a["Y"], a["scale"], P[5], 9, 64, 1,
                                        None) == ttt.ERR_INVALID_ARG


def rms_bwd(**kw):
    a = dict(R=P[0], w=P[1], dY=P[2], dR=P[3], eps=1e-6, dX=P[4], dw=P[5], rows=9, D=64, io=1,
             ws=P[6], wsb=BIG)
    a.update(kw)
    return ttt.lib().ttt_rmsnorm_bwd(a["R"], a["w"], a["dY"], a["dR"], a["eps"], a["dX"], a["dw"],
                                     a["rows"], a["D"], a["io"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=None), -1), (dict(dY=None), -1), (dict(dX=None), -1), (dict(R=P[0] + 2), -1),
    (dict(dw=P[5] + 2), -1), (dict(eps=0.0), -1), (dict(eps=1e-39), -1), (dict(rows=-2), -1), (dict(D=0), -1),
    (dict(io=9), -1), (dict(D=0x7fffffff), -1), (dict(dX=P[0]), -1), (dict(dX=P[2] + 16), -1), (dict(dX=P[3] + 16), -1),
    (dict(dX=P[1]), -1), (dict(dw=P[0]), -1), (dict(dw=P[1]), -1), (dict(dw=P[4]), -1),
    (dict(ws=None), -3), (dict(wsb=3), -3), (dict(ws=P[6] + 64), -3),
])
def test_rmsnorm_bwd_refuses(kw, status):
    assert rms_bwd(**kw) == status


def test_rmsnorm_empty_calls_do_nothing():
    L = ttt.lib()
    assert L.ttt_rmsnorm_fwd(None, None, None, 1e-6, None, None, 0, 64, 1, None) == ttt.OK
    assert L.ttt_rmsnorm_q8_fwd(None, None, None, 1e-6, None, None, None, 0, 64, 1, None) == ttt.OK
    assert L.ttt_rmsnorm_bwd(None, None, None, None, 1e-6, None, None, 0, 64, 1, None, 0,
                             None) == ttt.OK
    assert ttt.rmsnorm_bwd_workspace_bytes(-1, 64, 1) == 0


def clip(ranges, outs=True, norm=P[11], max_norm=1.0, eps=1e-6, ws=P[10], wsb=BIG, n=None):
    """ranges: (grad, out, elements, dtype) of each tensor."""
    k = len(ranges)
    g = (ctypes.c_void_p * k)(*[r[0] for r in ranges])
    o = (ctypes.c_void_p * k)(*[r[1] for r in ranges])
    s = (ctypes.c_longlong * k)(*[r[2] for r in ranges])
    t = (ctypes.c_int * k)(*[r[3] for r in ranges])
    return ttt.lib().ttt_clip_grad_norm(k if n is None else n, g, o if outs else None, s, t, max_norm,
                                        eps, norm, ws, wsb, None)


@pytest.mark.parametrize("ranges", [
    [(None, P[1], 4, 0)], [(P[0], None, 4, 0)], [(P[0], P[1], -1, 0)], [(P[0], P[1], 4, 2)],
    [(P[0] + 2, P[1], 4, 0)], [(P[0], P[1] + 1, 4, 1)], [(P[0], P[1], 1 << 62, 0)],
    [(P[0], P[0], 4, 0), (P[0], P[0], 4, 0)],              # the same gradient twice, in place
    [(P[0], P[2], 100, 0), (P[1], P[2] + 396, 4, 0)],      # outputs that share an element
    [(P[0], P[0] + 4, 100, 0)],                            # a shifted output
    [(P[0], P[2], 4, 0), (P[1], P[0], 4, 0)],              # an output on another's input
    [(P[0], P[1] - 396, 100, 0), (P[1], P[3], 4, 0)],      # reaching into another's input
    [(P[0], P[11] - 8, 4, 0)],                             # on the norm
    [(P[11] - 8, P[0], 4, 0)],
])
def test_clip_refuses_tensors(ranges):
    assert clip(ranges) == ttt.ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(norm=None), -1), (dict(norm=P[11] + 2), -1), (dict(max_norm=-1.0), -1),
    (dict(max_norm=math.nan), -1), (dict(eps=0.0), -1), (dict(eps=math.inf), -1), (dict(n=-1), -1),
    (dict(ws=None), -3), (dict(wsb=8), -3), (dict(ws=P[10] + 8), -3),
])
def test_clip_refuses_arguments(kw, status):
    assert clip([(P[0], P[1], 4, 0)], **kw) == status


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(1, 1, 4, 16)
    with pytest.raises(ValueError):
        ttt.gated_fwd(x, x)
    with pytest.raises(ValueError):
        ttt.gated_bwd(x, x, x)
    with pytest.raises(ValueError):
        ttt.gated_step(x, x, torch.zeros(1, 1, 16))
    with pytest.raises(ValueError):
        ttt.rmsnorm_fwd(x)
    with pytest.raises(ValueError):
        ttt.rmsnorm_q8_fwd(x)
    with pytest.raises(ValueError):
        ttt.rmsnorm_bwd(x, None, x)
    with pytest.raises(ValueError):
        ttt.clip_grad_norm([x], 1.0)
    with pytest.raises(ValueError):
        ttt.clip_grad_norm([], 1.0)
