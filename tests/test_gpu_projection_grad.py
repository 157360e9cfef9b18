"""GPU parity of the projections' gradients (flash_mca_gau_project_backward,
flash_mca_gau_output_backward) against the fp64 oracle (oracle/layer.py).

Bounds, element by element, with r = 2^-8 (half a step of bf16) and a sum of K
products in the tensor cores' fp32 accumulator off by at most K 2^-23 sum|a b|
(one rounding, or cut, a step): an output is off by its own rounding r |out|
and K 2^-23 sum|a b|.  dpre is rounded to bf16 and comes from pre (off by dz = d
2^-23 sum|x w|) through silu' (slope at most 1/2 in pre, fp32 evaluation within
2^-18): |dOut| (dz / 2 + 2^-18) + r |dpre|, which the products carry on.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import layer

from tests.test_gpu_parity import fm

pytestmark = pytest.mark.gpu

R = 2.0 ** -8 * 1.001
ACC = 2.0 ** -23
BF = torch.bfloat16


def rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(BF)


def np64(t):
    return t.double().cpu().numpy()


def status_ok(m):
    torch.cuda.synchronize()
    assert m.flash_mca_device_status()[0] == m.FMCA_OK


def product_bound(a, b, da, out):
    """Bound of a bf16 product a @ b whose a is off by da."""
    K = a.shape[1]
    return R * np.abs(out) + (da + K * ACC * (np.abs(a) + da)) @ np.abs(b)


def check_project(m, X, Wt, dU, dV, dZ, dX, dWt):
    x, w = np64(X), np64(Wt)
    rX, rW, dpre = layer.gau_project_backward(x, w, np64(dU), np64(dV), np64(dZ))
    up = np.abs(np.concatenate([np64(dU), np64(dV), np64(dZ)], 1))
    dz = x.shape[1] * ACC * (np.abs(x) @ np.abs(w).T)
    e = R * np.abs(dpre) + up * (dz / 2 + 2.0 ** -18)
    assert (np.abs(np64(dX) - rX) <= product_bound(dpre, w, e, rX)).all()
    assert (np.abs(np64(dWt) - rW) <= product_bound(dpre.T, x, e.T, rW)).all()


# one row, rows around the 64-token blocks and 128 / 256-row tiles, depths that
# are no multiple of 64, widths below, at and past a 256-column tile, products
# whose k axis is split (few tiles, many rows; few rows, many columns)
PROJECT = [(1, 64, 64, 64), (3, 8, 64, 64), (63, 72, 64, 64), (64, 768, 128, 128), (65, 520, 448, 64),
           (127, 256, 192, 256), (129, 248, 64, 128), (255, 264, 320, 64), (257, 1000, 128, 64),
           (1001, 520, 448, 64), (4100, 64, 64, 64), (40, 136, 1536, 128), (300, 768, 1536, 128)]


@pytest.mark.parametrize("M,d,e,s", PROJECT)
def test_project_backward(M, d, e, s):
    m = fm()
    X, Wt = rand((M, d), M + d).cuda(), rand((2 * e + s, d), e, d ** -0.5).cuda()
    up = [rand((M, k), 7 * M + i).cuda() for i, k in enumerate((e, e, s))]
    dX, dWt = m.gau_project_backward(X, Wt, *up)
    status_ok(m)
    check_project(m, X, Wt, *up, dX, dWt)
    again = m.gau_project_backward(X, Wt, *up)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dWt)


def test_project_backward_of_large_values():
    """pre far into both tails of the sigmoid: silu' is 0 or 1 there."""
    m = fm()
    X, Wt = rand((70, 64), 1, 30.0).cuda(), rand((192, 64), 2, 3.0).cuda()
    up = [rand((70, 64), 3 + i).cuda() for i in range(3)]
    dX, dWt = m.gau_project_backward(X, Wt, *up)
    check_project(m, X, Wt, *up, dX, dWt)


OUTPUT = [(1, 64, 64), (2, 8, 64), (77, 136, 64), (130, 1000, 320), (256, 1536, 768), (513, 264, 128),
          (5000, 72, 64), (64, 2048, 1024)]


@pytest.mark.parametrize("M,e,d", OUTPUT)
def test_output_backward(M, e, d):
    m = fm()
    Y, Wo, dOut = rand((M, e), M).cuda(), rand((d, e), e, e ** -0.5).cuda(), rand((M, d), d).cuda()
    dY, dWo = m.gau_output_backward(Y, Wo, dOut)
    status_ok(m)
    y, w, g = np64(Y), np64(Wo), np64(dOut)
    rY, rW = layer.gau_output_backward(y, w, g)
    assert (np.abs(np64(dY) - rY) <= product_bound(g, w, 0 * g, rY)).all()
    assert (np.abs(np64(dWo) - rW) <= product_bound(g.T, y, 0 * g.T, rW)).all()


def test_outputs_in_larger_buffers_and_half_aligned():
    """Rows behind the last stay; outputs that start on a 16-byte boundary only."""
    m = fm()
    M, e, d = 70, 136, 64
    Y, Wo, dOut = rand((M, e), 1).cuda(), rand((d, e), 2).cuda(), rand((M, d), 3).cuda()
    ref = m.gau_output_backward(Y, Wo, dOut)
    ws = torch.empty(m.flash_mca_gau_output_backward_workspace_bytes(M, e, d), dtype=torch.uint8,
                     device="cuda")
    by, bw = [torch.full((8 + n * e + 512,), 5.0, dtype=BF, device="cuda") for n in (M, d)]
    dY, dW = by[8:8 + M * e].view(M, e), bw[8:8 + d * e].view(d, e)
    m.flash_mca_gau_output_backward(Y, Wo, dOut, dY, dW, ws)
    torch.cuda.synchronize()
    assert torch.equal(dY, ref[0]) and torch.equal(dW, ref[1])
    for b, n in ((by, M), (bw, d)):
        assert (b[:8] == 5.0).all() and (b[8 + n * e:] == 5.0).all()


def test_streams_and_two_graphs():
    m = fm()
    M, d, e, s = 200, 128, 128, 64
    X, Wt = rand((M, d), 1).cuda(), rand((2 * e + s, d), 2, d ** -0.5).cuda()
    up = [rand((M, k), 3 + i).cuda() for i, k in enumerate((e, e, s))]
    ref = m.gau_project_backward(X, Wt, *up)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [m.gau_project_backward(X, Wt, *up, stream=st) for st in side for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, ref))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = m.gau_project_backward(X, Wt, *up)
        graphs.append((g, out))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for _, out in graphs for a, b in zip(out, ref))


def test_refusals():
    m = fm()
    X, Wt, g = rand((8, 64), 1).cuda(), rand((192, 64), 2).cuda(), rand((8, 64), 3).cuda()
    for bad in (lambda: m.gau_project_backward(X, Wt[:128], g, g, g),
                lambda: m.gau_project_backward(X, Wt, g, g[:4], g),
                lambda: m.gau_project_backward(X.float(), Wt, g, g, g),
                lambda: m.gau_project_backward(X, Wt, g, g.cpu(), g),
                lambda: m.gau_output_backward(X, Wt[:64].t(), g),
                lambda: m.gau_output_backward(X, Wt, g)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: m.gau_project_backward(X[:0], Wt, g[:0], g[:0], g[:0]),
                lambda: m.gau_project_backward(X, Wt[:96], g[:, :32].contiguous(),
                                               g[:, :32].contiguous(), g[:, :32].contiguous()),
                lambda: m.gau_output_backward(X, Wt[:32], g[:, :32].contiguous())):
        with pytest.raises(m.FmcaError):
            bad()


# both sides of the sizes up to which a product goes in 128 x 128 tiles, and the
# two launches of a call on different ones
TILES = [(100, 64, 9664, 64), (100, 64, 9728, 64), (1200, 512, 960, 64), (1001, 2000, 448, 64),
         (300, 2600, 192, 64), (300, 2696, 192, 64)]


@pytest.mark.parametrize("M,d,e,s", TILES)
def test_project_backward_in_either_tile(M, d, e, s):
    test_project_backward(M, d, e, s)


@pytest.mark.parametrize("M,e,d", [(1000, 1152, 1024), (1000, 1224, 1024), (129, 4864, 384),
                                   (129, 4872, 384)])
def test_output_backward_in_either_tile(M, e, d):
    test_output_backward(M, e, d)
