"""GPU parity of flash_mca_layer_norm and its backward pass against the fp64
oracle (oracle/layer.py) on the same inputs.

Bounds, with u = 2^-24 (half a step of fp32) and r the half step of the I/O
type (2^-8 bf16, u fp32).  A row's sums take at most 32 additions in a thread,
5 in a warp and 8 across a block: 45 roundings, so the mean is off by at most
45 u max|h|, and rstd by a factor 1 + 30 u.  With A = rstd max|h| of the row
that puts xhat off by at most (45 + 2 * 32) u A < 128 u A, and y by 128 u (A |w|
+ |b|) + r |y|.  In the backward pass, with T = max|t| and X = max|xhat|:
mean(t) and mean(t xhat) are at most T and off by 45 u T (+ T times xhat's
error); dx is off by at most rstd T (1 + X) (128 u + 2 * 128 u A) + r |dx|.  dw:
sum|dy| times xhat's error, and 64 roundings of sums of |dy xhat|.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import layer

from tests.test_gpu_parity import fm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def half_step(dt):
    return torch.finfo(dt).eps / 2


def make(M, d, dt, seed, residual, shift=0.3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (1.5 * n(M, d) + shift).to(dt)
    res = (0.7 * n(M, d)).to(dt) if residual else None
    w, b = 1 + 0.2 * n(d), 0.2 * n(d)
    return x, res, w, b, n(M, d).to(dt), (n(M, d).to(dt) if residual else None)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def np64(t):
    return t.double().cpu().numpy()


def check_forward(h, w, b, y, mean, rstd, dt, eps=EPS):
    ry, xhat, rmean, rrstd = layer.layer_norm(np64(h), np64(w), np64(b), eps)
    top = np.abs(np64(h)).max(1)
    A = (rrstd * top)[:, None]
    bound = 128 * U * (A * np.abs(np64(w)) + np.abs(np64(b))) + half_step(dt) * np.abs(ry) * 1.01
    assert (np.abs(np64(y) - ry) <= bound).all()
    assert (np.abs(np64(mean) - rmean) <= 46 * U * top).all()
    assert (np.abs(np64(rstd) - rrstd) <= 32 * U * rrstd * (1 + A[:, 0])).all()
    return A


def check_backward(dy, h, w, dh, dx, dw, db, dt, eps=EPS):
    rdx, rdw, rdb = layer.layer_norm_backward(np64(dy), np64(h), np64(w), eps,
                                              None if dh is None else np64(dh))
    _, xhat, _, rrstd = layer.layer_norm(np64(h), np64(w), np64(w), eps)
    A = rrstd * np.abs(np64(h)).max(1)
    T = np.abs(np64(dy) * np64(w)).max(1)
    X = np.abs(xhat).max(1)
    b = rrstd * T * (1 + X) * (128 * U + 256 * U * A)
    bound = b[:, None] + half_step(dt) * np.abs(rdx) * 1.01 + \
        (0 if dh is None else 2 * U * np.abs(np64(dh)))
    assert (np.abs(np64(dx) - rdx) <= bound).all()
    g = np.abs(np64(dy))
    assert (np.abs(np64(dw) - rdw) <= (g * (128 * U * A)[:, None]).sum(0)
            + 64 * U * (g * np.abs(xhat)).sum(0)).all()
    assert (np.abs(np64(db) - rdb) <= 64 * U * g.sum(0)).all()


# every vector width (16 bytes, 4 bytes, single elements), elements a thread
# (8 .. 32), warp and block rows, and both sides of their borders
SIZES = [(1, 1), (1, 768), (3, 7), (64, 768), (37, 255), (9, 256), (8, 257), (50, 512), (11, 513),
         (5, 770), (17, 1001), (4, 1024), (6, 1025), (7, 1032), (3, 2050), (5, 4096), (3, 6150),
         (2, 8191), (3, 8192), (3001, 128), (2500, 33)]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,d", SIZES)
def test_layer_norm(M, d, dt):
    m = fm()
    residual = (M + d) % 2 == 0
    x, res, w, b, dy, dh = cuda(*make(M, d, dt, 100 * M + d, residual))
    y, h, mean, rstd = m.layer_norm(x, w, b, EPS, residual=res)
    if residual:  # the sum of two values of the type, rounded once
        assert torch.equal(h, (x.double() + res.double()).to(dt))
    else:
        assert h is x
    check_forward(h, w, b, y, mean, rstd, dt)
    dx, dw, db = m.layer_norm_backward(dy, h, w, mean, rstd, dh)
    check_backward(dy, h, w, dh, dx, dw, db, dt)


def test_rows_that_are_constant_large_or_tiny():
    m = fm()
    d = 768
    x = torch.randn(6, d, generator=torch.Generator().manual_seed(1))
    x[0] = 3.0                       # no deviation: rstd = 1 / sqrt(eps)
    x[1] = 0.0
    x[2] *= 1e15                     # squares near the top of fp32's range
    x[3] *= 1e-20                    # squares below its smallest number
    x[4] += 1000.0                   # a mean far from 0
    w, b = torch.ones(d), torch.zeros(d)
    x, w, b = cuda(x, w, b)
    y, h, mean, rstd = m.layer_norm(x, w, b, EPS)
    check_forward(h, w, b, y, mean, rstd, F32)
    assert torch.equal(y[1], torch.zeros_like(y[1]))


def test_nan_and_infinity_stay_in_their_rows():
    m = fm()
    x, _, w, b, dy, _ = cuda(*make(9, 320, BF, 4, False))
    ref = m.layer_norm(x, w, b)
    bad = x.clone()
    bad[2, 5], bad[7, 0] = float("nan"), float("inf")
    y, _, mean, rstd = m.layer_norm(bad, w, b)
    keep = [0, 1, 3, 4, 5, 6, 8]
    assert torch.equal(y[keep], ref[0][keep])
    assert torch.isnan(y[[2, 7]]).all()


def test_residual_updated_in_place_and_rows_behind_the_last():
    m = fm()
    x, res, w, b, dy, dh = cuda(*make(33, 776, BF, 5, True))
    y0, h0, mean, rstd = m.layer_norm(x, w, b, EPS, residual=res)
    # outputs inside larger buffers: what lies behind the last row stays
    big = [torch.full((40, 776), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    hb = torch.full((40, 776), 9.0, dtype=BF, device="cuda")
    hb[:33] = x
    m.flash_mca_layer_norm(hb[:33], res, w, b, hb[:33], big[0][:33], None, None, EPS)
    assert torch.equal(hb[:33], h0) and torch.equal(big[0][:33], y0)
    assert (hb[33:] == 9.0).all() and (big[0][33:] == 7.0).all()
    rr = res.clone()
    m.flash_mca_layer_norm(x, rr, w, b, rr, big[1][:33], None, None, EPS)
    assert torch.equal(rr, h0) and torch.equal(big[1][:33], y0)


def test_leading_dimensions_streams_and_replays():
    m = fm()
    x, res, w, b, dy, dh = cuda(*make(24, 768, BF, 6, True))
    y, h, mean, rstd = m.layer_norm(x, w, b, EPS, residual=res)
    dx, dw, db = m.layer_norm_backward(dy, h, w, mean, rstd, dh)
    y3, h3, mean3, rstd3 = m.layer_norm(x.view(2, 12, 768), w, b, EPS, residual=res.view(2, 12, 768))
    assert y3.shape == (2, 12, 768) and mean3.shape == (2, 12)
    assert torch.equal(y3.view(24, 768), y) and torch.equal(rstd3.view(24), rstd)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ys, hs, ms, rs = m.layer_norm(x, w, b, EPS, residual=res, stream=side)
    gs = m.layer_norm_backward(dy, hs, w, ms, rs, dh, stream=side)
    side.synchronize()
    assert torch.equal(ys, y) and all(torch.equal(a, c) for a, c in zip(gs, (dx, dw, db)))
    # two graphs captured over the same inputs, replayed in turn
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            yg, hg, mg, rg = m.layer_norm(x, w, b, EPS, residual=res)
            out = m.layer_norm_backward(dy, hg, w, mg, rg, dh)
        graphs.append((g, yg, out))
    for _ in range(2):
        for g, yg, out in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, yg, out in graphs:
        assert torch.equal(yg, y) and all(torch.equal(a, c) for a, c in zip(out, (dx, dw, db)))


def test_more_rows_than_32_bits_of_elements_reach():
    """Row offsets past 2^31 elements: the last rows of a tall matrix."""
    m = fm()
    M, d = (1 << 31) // 1024 + 100, 1024
    x = torch.zeros(M, d, dtype=BF, device="cuda")
    tail = make(200, d, BF, 7, False)[0].cuda()
    x[-200:] = tail
    w, b = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    y = torch.empty_like(x)
    m.flash_mca_layer_norm(x, None, w, b, None, y, None, None, EPS)
    ref = m.layer_norm(tail, w, b, EPS)[0]
    assert torch.equal(y[-200:], ref)
    assert (y[:4] == 0).all()


def test_refusals():
    m = fm()
    x, res, w, b, dy, dh = cuda(*make(4, 64, BF, 8, True))
    for bad in (lambda: m.layer_norm(x[:0], w, b), lambda: m.layer_norm(x.t(), w[:4], b[:4]),
                lambda: m.layer_norm(x, w.to(BF), b), lambda: m.layer_norm(x, w[:32], b),
                lambda: m.layer_norm(x, w, b, residual=res.float()),
                lambda: m.layer_norm(x, w, b, residual=res[:2]),
                lambda: m.layer_norm(x, w, b.cpu()),
                lambda: m.flash_mca_layer_norm(x, res, w, b, None, torch.empty_like(x), None, None)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        m.layer_norm(x.half(), w, b)
    big = torch.zeros(2, 8200, device="cuda")
    for bad in (lambda: m.layer_norm(big, big[0], big[1]),
                lambda: m.layer_norm(x, w, b, eps=-1.0),
                lambda: m.flash_mca_layer_norm(x, None, w, b, None, x, None, None)):  # y is x
        with pytest.raises(m.FmcaError):
            bad()


def test_outputs_are_tensors_of_their_own():
    """What the wrappers return: fresh, contiguous, aligned, and apart from each
    other (writing one leaves the rest)."""
    m = fm()
    x, res, w, b, dy, dh = cuda(*make(7, 65, F32, 9, True))
    y, h, mean, rstd = m.layer_norm(x, w, b, residual=res)
    dx, dw, db = m.layer_norm_backward(dy, h, w, mean, rstd, dh)
    outs = [y, h, mean, rstd, dx, dw, db]
    assert [tuple(t.shape) for t in outs] == [(7, 65), (7, 65), (7,), (7,), (7, 65), (65,), (65,)]
    keep = [t.clone() for t in outs]
    for i, t in enumerate(outs):
        assert t.is_contiguous() and t.data_ptr() % 16 == 0 and not t.requires_grad
        t.fill_(-1.0)
        assert all(torch.equal(a, c) for a, c in zip(outs[i + 1:], keep[i + 1:]))
        assert (t == -1.0).all()


# rows of several warps, and several rows a group, at both sides of the number of
# rows up to which the backward pass spreads a row over more warps
MANY = [(8192, 640, BF), (8193, 640, BF), (3000, 776, BF), (4099, 1002, BF), (4099, 1001, BF),
        (4099, 1001, F32), (2600, 201, F32), (2000, 2001, F32), (1, 776, BF), (5, 640, BF)]


@pytest.mark.parametrize("M,d,dt", MANY, ids=lambda v: str(v).removeprefix("torch."))
@pytest.mark.parametrize("residual", [False, True])
def test_backward_of_many_rows(M, d, dt, residual):
    m = fm()
    x, _, w, b, dy, dh = cuda(*make(M, d, dt, M + d, residual))
    _, h, mean, rstd = m.layer_norm(x, w, b, EPS)
    dx, dw, db = m.layer_norm_backward(dy, h, w, mean, rstd, dh)
    check_backward(dy, h, w, dh, dx, dw, db, dt)
    again = m.layer_norm_backward(dy, h, w, mean, rstd, dh)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("M,d,dt", [(5000, 256, BF), (5000, 1536, BF), (3000, 2048, BF),
                                    (5000, 256, F32), (1000, 1028, F32)],
                         ids=lambda v: str(v).removeprefix("torch."))
def test_backward_with_three_blocks_an_sm(M, d, dt):
    test_backward_of_many_rows(M, d, dt, True)


# bf16 rows of odd lengths, each starting somewhere else within 16 bytes, come
# whole: up to the longest, the last row ending with the array, rows behind it
WHOLE = [(1, 1), (7, 3), (900, 17), (2000, 255), (1300, 257), (700, 1023), (1301, 1025),
         (311, 4001), (200, 8191)]


@pytest.mark.parametrize("M,d", WHOLE)
@pytest.mark.parametrize("residual", [False, True])
def test_backward_of_rows_that_start_anywhere(M, d, residual):
    m = fm()
    x, _, w, b, dy, dh = cuda(*make(M, d, BF, M + d, residual))
    _, h, mean, rstd = m.layer_norm(x, w, b, EPS)
    want = m.layer_norm_backward(dy, h, w, mean, rstd, dh)
    check_backward(dy, h, w, dh, *want, BF)
    # the same rows ahead of others that hold NaN
    more = torch.full((M + 1, d), float("nan"), device="cuda", dtype=BF)
    parts = [None if t is None else more.clone() for t in (dy, h, dh)]
    for p, t in zip(parts, (dy, h, dh)):
        if t is not None:
            p[:M] = t
    got = m.layer_norm_backward(parts[0][:M], parts[1][:M], w, mean, rstd,
                                None if dh is None else parts[2][:M])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("M,d,dt", [(700, 2049, F32), (500, 2052, F32), (300, 4096, F32),
                                    (300, 4095, F32), (200, 4097, F32), (100, 5700, F32),
                                    (700, 2050, BF), (300, 4094, BF), (200, 4098, BF),
                                    (500, 2056, BF), (600, 511, F32), (600, 513, F32),
                                    (600, 510, BF), (600, 514, BF), (600, 511, BF)],
                         ids=lambda v: str(v).removeprefix("torch."))
def test_long_rows_and_quarter_blocks(M, d, dt):
    test_layer_norm(M, d, dt)
    test_backward_of_many_rows(M, d, dt, True)
