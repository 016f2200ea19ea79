"""GPU parity of the gradient norm and clipping with its fp64 form.  The norm is a sum in fp64
rounded to fp32 (2^-24 relative, and far less of its own); an output is one fp32 factor (2^-24), one
product (2^-24) and the rounding to its type."""
import numpy as np
import pytest

import block_ref as ref
from gpu_helpers import say
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    return torch.device("cuda:0")


def make(dev, sizes, io, seed, scale=0.01):
    """A tensor of each size; io "mixed": every other one bf16."""
    import torch
    gen = torch.Generator(device="cpu").manual_seed(seed)
    out = []
    for k, n in enumerate(sizes):
        bf = io == "bf16" or (io == "mixed" and k % 2 == 0)
        out.append((scale * torch.randn(n, generator=gen)).to(dev, torch.bfloat16 if bf else torch.float32))
    return out


def np64(t):
    return t.double().cpu().numpy()


def kind(t):
    return "f32" if t.element_size() == 4 else "bf16"


def check(grads, outs, norm, max_norm, eps=1e-6):
    want, n = ref.clip([np64(g) for g in grads], max_norm, eps)
    say("  norm %.6g" % n)
    assert ref.within(np64(norm), np.array([n]), n * 2 * ref.U, "f32")[0]
    for k, (o, v) in enumerate(zip(outs, want)):
        ok, worst = ref.within(np64(o), v, np.abs(v) * 3 * ref.U, kind(o))
        assert ok, (k, worst)


@pytest.mark.parametrize("io", ["bf16", "f32", "mixed"])
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [7, 8, 9, 16, 17, 1000], [4096, 16384, 16385, 100001],
                                   [1 << 20, 3, 300000], [257] * 61])
def test_sizes(dev, sizes, io):
    say("case", sizes[:6], io)
    grads = make(dev, sizes, io, len(sizes))
    for max_norm in (1e-3, 0.05, 1e9, float("inf"), 0.0):
        outs, norm = ttt.clip_grad_norm(grads, max_norm)
        check(grads, outs, norm, max_norm)


@pytest.mark.parametrize("n", [63, 64, 65, 100, 128, 129, 400, 1000])
def test_many_tensors(dev, n):
    say("case n", n)
    grads = make(dev, [(k * 37) % 500 for k in range(n)], "mixed", n)
    outs, norm = ttt.clip_grad_norm(grads, 0.01)
    check(grads, outs, norm, 0.01)


@pytest.mark.parametrize("max_norm", [0.01, 1e9])
def test_in_place(dev, max_norm):
    import torch
    grads = make(dev, [5000, 3, 70000, 0, 129], "mixed", 3)
    outs, norm = ttt.clip_grad_norm(grads, max_norm)
    same = [g.clone() for g in grads]
    got, norm2 = ttt.clip_grad_norm(same, max_norm, outs=same)
    assert torch.equal(norm, norm2)
    for a, b in zip(outs, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_alignment(dev, io, shift):
    """Tensors that start anywhere in their buffer, outputs elsewhere; what is around them stays."""
    import torch
    big = make(dev, [20000, 20000], io, 5)
    grads = [big[0][shift:shift + 9001], big[1][8:8 + 777]]
    bufs = [torch.full((20000,), 7.0, dtype=big[0].dtype, device=dev) for _ in range(2)]
    outs = [bufs[0][2 * shift:2 * shift + 9001], bufs[1][shift:shift + 777]]
    got, norm = ttt.clip_grad_norm(grads, 0.05, outs=outs)
    check(grads, got, norm, 0.05)
    for b, at, n in ((bufs[0], 2 * shift, 9001), (bufs[1], shift, 777)):
        assert (b[:at] == 7).all() and (b[at + n:] == 7).all()


def test_norm_alone(dev):
    import torch
    grads = make(dev, [1000, 70], "mixed", 7)
    import ctypes
    norm = torch.zeros(1, device=dev)
    ws = torch.empty(ttt.clip_workspace_bytes(), dtype=torch.uint8, device=dev)
    gp = (ctypes.c_void_p * 2)(*[g.data_ptr() for g in grads])
    sz = (ctypes.c_longlong * 2)(1000, 70)
    dt = (ctypes.c_int * 2)(1, 0)
    assert ttt.lib().ttt_clip_grad_norm(2, gp, None, sz, dt, 1.0, 1e-6, norm.data_ptr(), ws.data_ptr(),
                                        ws.numel(), torch.cuda.current_stream().cuda_stream) == ttt.OK
    check(grads, [], norm, 1.0)


def test_nothing(dev):
    import torch
    norm = torch.full((1,), 5.0, device=dev)
    outs, norm = ttt.clip_grad_norm([], 1.0, norm=norm)
    assert outs == [] and norm.item() == 0.0
    g = [torch.zeros(100, device=dev), torch.zeros(0, device=dev)]
    outs, norm = ttt.clip_grad_norm(g, 1.0)
    assert norm.item() == 0.0 and (outs[0] == 0).all()


def test_values_whose_squares_leave_fp32(dev):
    import torch
    for v in (1e30, 1e-30):
        g = [torch.full((1000,), v, device=dev), torch.full((24,), -v, device=dev)]
        outs, norm = ttt.clip_grad_norm(g, 1.0)
        check(g, outs, norm, 1.0)


def test_what_is_not_finite(dev):
    import torch
    g = make(dev, [300, 40], "f32", 9)
    g[1][7] = float("nan")
    outs, norm = ttt.clip_grad_norm(g, 1.0)
    assert torch.isnan(norm).all() and all(torch.isnan(o).all() for o in outs)
    g[1][7] = float("inf")
    outs, norm = ttt.clip_grad_norm(g, 1.0)
    assert torch.isinf(norm).all() and (outs[0] == 0).all() and torch.isnan(outs[1][7])


def test_same_bits_every_time(dev):
    import torch
    g = make(dev, [700001, 3, 1 << 20], "mixed", 11)
    outs, norm = ttt.clip_grad_norm(g, 0.5)
    ws = torch.empty(ttt.clip_workspace_bytes(), dtype=torch.uint8, device=dev)
    for k in range(5):
        ws.fill_(63 * k)
        o2, n2 = ttt.clip_grad_norm(g, 0.5, workspace=ws)
        assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(outs, o2))


def test_offsets_past_32_bits(dev):
    import torch
    n = (1 << 31) + 4099
    g = [torch.zeros(n, dtype=torch.bfloat16, device=dev)]
    g[0][-5:] = 3.0
    g[0][0] = 4.0
    outs, norm = ttt.clip_grad_norm(g, 1.0, outs=g)
    want = np.sqrt(5 * 9 + 16.0)
    assert abs(norm.item() - want) <= 2 * want * ref.U
    assert abs(outs[0][-1].item() - 3 / want) <= 3 / want * 2.0 ** -8
    assert outs[0][n // 2].item() == 0
