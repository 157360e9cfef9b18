"""GPU parity of the vocabulary loss and its gradients (flash_mca_vocab_loss,
flash_mca_vocab_loss_backward) against the fp64 oracle (oracle/layer.py; at the
larger sizes the same formulas as torch fp64 operations on the GPU).

Bounds, with r = 2^-8 (half a step of bf16) and a sum of K products in the
tensor cores' fp32 accumulator off by at most K 2^-23 sum|a b|: a logit is off
by dz = d 2^-23 sum|x w| (D: the row's largest), lse by D + 2^-20 (1 + |lse|)
(the sum's own roundings are relative and go through the logarithm), the loss
by 2 D + 2^-20 (1 + |lse|).  A probability is off by a factor 2 D + 2^-19 (1 +
|lse|), the bf16 entries of (p - onehot) g by that and r; the products carry
both on and the gradients are rounded once more.
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


def make(M, V, d, keep, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(M, d, generator=g).to(BF)
    W = (scale * d ** -0.5 * torch.randn(V, d, generator=g)).to(BF)
    t = torch.randint(0, V, (M,), generator=g)
    drop = torch.rand(M, generator=g) >= keep
    t[drop] = torch.tensor([-100, -1, V, 1 << 40])[torch.randint(0, 4, (M,), generator=g)][drop]
    dloss = torch.rand(M, generator=g) + 0.1
    dloss[torch.rand(M, generator=g) < 0.3] *= -1
    return X.cuda(), W.cuda(), t.cuda(), dloss.cuda()


def reference(X, W, t, dloss):
    """(loss, lse, dX, dW) and their bounds, in fp64 on the inputs' device."""
    x, w, g = X.double(), W.double(), dloss.double()
    M, d = x.shape
    V = w.shape[0]
    has = (t >= 0) & (t < V)
    x = torch.where(has[:, None], x, torch.zeros_like(x))
    g = torch.where(has, g, torch.zeros_like(g))
    at = torch.where(has, t, torch.zeros_like(t))
    z = x @ w.T
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, at[:, None])[:, 0]
    D = (d * ACC * (x.abs() @ w.abs().T)).amax(1)
    del_loss = 2 * D + 2.0 ** -20 * (1 + lse.abs())
    p = torch.exp(z - lse[:, None])
    q = p.clone()
    q[torch.arange(M, device=q.device), at] -= 1.0
    q *= g[:, None]
    dX, dW = q @ w, q.T @ x
    e = R * q.abs() + p * g.abs()[:, None] * (2 * D + 2.0 ** -19 * (1 + lse.abs()))[:, None]
    bX = R * dX.abs() + (e + V * ACC * (q.abs() + e)) @ w.abs()
    bW = R * dW.abs() + (e + M * ACC * (q.abs() + e)).T @ x.abs()
    zero = torch.zeros_like(lse)
    return ((torch.where(has, loss, zero), del_loss), (torch.where(has, lse, zero), del_loss),
            (dX, bX), (dW, bW))


def run(m, X, W, t, dloss):
    loss, lse = m.vocab_loss(X, W, t)
    dX, dW = m.vocab_loss_backward(X, W, t, lse, dloss)
    return loss, lse, dX, dW


def check(m, X, W, t, dloss):
    got = run(m, X, W, t, dloss)
    torch.cuda.synchronize()
    assert m.flash_mca_device_status()[0] == m.FMCA_OK
    for name, a, (ref, bound) in zip(("loss", "lse", "dX", "dW"), got, reference(X, W, t, dloss)):
        off = (a.double() - ref).abs()
        bad = ~(off <= bound)
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside, " \
                              f"largest {float(off[bad].max()):.3e}"
    return got


# rows around 32, 64, 128, 256; vocabularies below, at and past a tile; depths
# that are no multiple of 64; few rows of a long vocabulary and many of a short
# one (split depths)
SIZES = [(1, 1, 8), (1, 2, 64), (2, 300, 64), (31, 256, 72), (33, 255, 64), (64, 257, 136),
         (65, 511, 256), (127, 1000, 64), (128, 513, 768), (129, 769, 520), (200, 128, 64),
         (256, 2048, 256), (257, 129, 1000), (37, 8191, 256), (5, 40001, 64), (3000, 100, 64),
         (9000, 17, 96), (700, 5003, 200),
         (512, 600, 64), (513, 600, 64), (400, 16000, 768)]  # the rows' two forms meet here


@pytest.mark.parametrize("keep", [1.0, 0.3])
@pytest.mark.parametrize("M,V,d", SIZES)
def test_vocab_loss(M, V, d, keep):
    check(fm(), *make(M, V, d, keep, M + V + d))


def test_reference_is_the_oracle():
    X, W, t, dloss = make(40, 30, 16, 0.6, 9)
    ref = [r[0].cpu().numpy() for r in reference(X, W, t, dloss)]
    a = [v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy()
         for v in (X, W, t, dloss)]
    want = layer.vocab_loss(*a[:3]) + layer.vocab_loss_backward(*a)
    for r, w in zip(ref, want):
        np.testing.assert_allclose(r, w, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("M,V,d,keep", [
    (4200, 40100, 64, 1.0),    # two pieces of the vocabulary
    (8200, 33000, 64, 0.9),
    (8200, 33000, 64, 0.15),   # two by the row count, one by the rows that have a target
    (70000, 2100, 16, 1.0),    # pieces of few columns: dW's depth split in each
    (70000, 2100, 16, 0.02),
])
def test_vocabulary_in_pieces(M, V, d, keep):
    check(fm(), *make(M, V, d, keep, M + V))


def test_sharp_and_flat_rows():
    """Probabilities of 1 and of 1 / V, logits of +-200, equal logits."""
    m = fm()
    X, W, t, dloss = make(96, 700, 64, 1.0, 21)
    X[:32] *= 100.0
    X[32:64] = 0.0
    t[:16] = (X[:16].float() @ W.float().T).argmax(1)
    check(m, X, W, t, dloss)


@pytest.mark.parametrize("M", [900, 300, 90])
def test_rows_without_target_reach_nothing(M):
    """NaN and infinities in ignored rows of X, and in their dloss."""
    m = fm()
    X, W, t, dloss = make(M, 1000, 128, 0.5, 31)
    clean = run(m, X, W, t, dloss)
    out = (t < 0) | (t >= 1000)
    X2, g2 = X.clone(), dloss.clone()
    X2[out] = float("nan")
    X2[out.nonzero()[0]] = float("inf")
    g2[out] = float("nan")
    dirty = run(m, X2, W, t, g2)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
    assert (dirty[0][out] == 0).all() and (dirty[1][out] == 0).all() and (dirty[2][out] == 0).all()


@pytest.mark.parametrize("M", [1, 64, 300, 1000])
def test_no_row_has_a_target(M):
    m = fm()
    X, W, t, dloss = make(M, 500, 64, 1.0, 41)
    t[:] = -100
    X[:] = float("nan")
    for a in run(m, X, W, t, dloss):
        assert (a == 0).all()


@pytest.mark.parametrize("M", [600, 200, 100])
def test_nan_stays_in_its_row_and_weights_of_zero(M):
    m = fm()
    X, W, t, dloss = make(M, 600, 64, 1.0, 51)
    ref = run(m, X, W, t, dloss)
    X2 = X.clone()
    X2[17, 3] = float("nan")
    loss, lse, dX, dW = run(m, X2, W, t, dloss)
    keep = torch.arange(M, device="cuda") != 17
    assert torch.isnan(loss[17]) and torch.isnan(dX[17]).all() and torch.isnan(dW).all()
    assert torch.equal(loss[keep], ref[0][keep]) and torch.equal(dX[keep], ref[2][keep])
    for a in m.vocab_loss_backward(X, W, t, ref[1], torch.zeros_like(dloss)):
        assert (a == 0).all()
    # rows with an infinite weight: the others keep finite gradients
    g2 = dloss.clone()
    g2[5] = float("inf")
    dX, dW = m.vocab_loss_backward(X, W, t, ref[1], g2)
    keep = torch.arange(M, device="cuda") != 5
    assert torch.isfinite(dX[keep]).all() and not torch.isfinite(dX[5]).any()


@pytest.mark.parametrize("M", [600, 150, 128])
def test_tiny_and_huge_weights_scale_the_gradients(M):
    """dloss times a power of two gives the gradients times it, bit for bit
    (no overflow or underflow in between)."""
    m = fm()
    X, W, t, dloss = make(M, 400, 64, 0.8, 61)
    _, lse = m.vocab_loss(X, W, t)
    base = m.vocab_loss_backward(X, W, t, lse, dloss)
    for k in (-60, 60):
        got = m.vocab_loss_backward(X, W, t, lse, dloss * 2.0 ** k)
        assert all(torch.equal(a.double(), b.double() * 2.0 ** k) for a, b in zip(got, base))


def test_same_bits_again_on_streams_and_behind_the_last_row():
    m = fm()
    X, W, t, dloss = make(333, 3001, 136, 0.7, 71)
    ref = run(m, X, W, t, dloss)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for st in streams:
            loss, lse = m.vocab_loss(X, W, t, stream=st)
            got.append((loss, lse) + m.vocab_loss_backward(X, W, t, lse, dloss, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, ref))
    big = [torch.full((400,), 3.0, device="cuda") for _ in range(2)]
    bx = torch.full((400, 136), 3.0, dtype=BF, device="cuda")
    bw = torch.full((3100, 136), 3.0, dtype=BF, device="cuda")
    ws = torch.empty(max(m.flash_mca_vocab_loss_workspace_bytes(333, 3001, 136),
                         m.flash_mca_vocab_loss_backward_workspace_bytes(333, 3001, 136)),
                     dtype=torch.uint8, device="cuda").fill_(255)  # NaN wherever it is read
    m.flash_mca_vocab_loss(X, W, t, big[0][:333], big[1][:333], ws)
    m.flash_mca_vocab_loss_backward(X, W, t, big[1][:333], dloss, bx[:333], bw[:3001], ws)
    torch.cuda.synchronize()
    for a, b, n in zip((*big, bx, bw), ref, (333, 333, 333, 3001)):
        assert torch.equal(a[:n], b) and (a[n:] == 3.0).all()


@pytest.mark.parametrize("M", [800, 500, 77])
def test_captured_calls_follow_the_targets(M):
    """Two graphs over the same inputs; the targets change between replays, so
    that the number of rows that take part does."""
    m = fm()
    X, W, t, dloss = make(M, 1500, 64, 1.0, 81)
    targets = [make(M, 1500, 64, k, 82)[2] for k in (1.0, 0.4, 0.0, 0.7)]
    refs = [run(m, X, W, v, dloss) for v in targets]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(m, X, W, t, dloss)
        graphs.append((g, out))
    for v, ref in zip(targets, refs):
        t.copy_(v)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_gradients_are_differences():
    """Along random directions: the change of the summed loss in X and in W."""
    m = fm()
    X, W, t, dloss = make(128, 300, 64, 0.8, 91, scale=1.0)
    _, lse = m.vocab_loss(X, W, t)
    dX, dW = m.vocab_loss_backward(X, W, t, lse, dloss)

    def total(x, w):
        (loss, _), *_ = reference(x, w, t, dloss)
        return float((loss * torch.where(loss != 0, dloss.double(), loss)).sum())
    g = torch.Generator(device="cuda").manual_seed(1)
    for which, grad in ((0, dX), (1, dW)):
        for _ in range(3):
            base = (X.double(), W.double())
            v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-4
            ends = []
            for sgn in (h, -h):
                a = list(base)
                a[which] = a[which] + sgn * v
                ends.append(total(*a))
            slope = (ends[0] - ends[1]) / (2 * h)
            # both roundings (2^-8 of each entry) and the difference's h^2 term
            bound = 2 * R * float((grad.double() * v).abs().sum()) + 1e-4
            assert abs(slope - float((grad.double() * v).sum())) <= bound


def test_refusals():
    m = fm()
    X, W, t, dloss = make(8, 20, 64, 1.0, 1)
    lse = torch.zeros(8, device="cuda")
    for bad in (lambda: m.vocab_loss(X[0], W, t),                       # not a matrix
                lambda: m.vocab_loss(X, W[:, :56], t),                  # widths differ
                lambda: m.vocab_loss(X, W.t().contiguous().t(), t),     # not contiguous
                lambda: m.vocab_loss(X, W, t.int()),
                lambda: m.vocab_loss(X, W, t[:7]),
                lambda: m.vocab_loss(X, W, t.cpu()),
                lambda: m.vocab_loss(X.half(), W.half(), t),
                lambda: m.vocab_loss_backward(X, W, t, lse[:4], dloss),
                lambda: m.vocab_loss_backward(X, W, t, lse, dloss.double()),
                lambda: m.flash_mca_vocab_loss(X, W, t, lse, lse[:4], lse.byte())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: m.vocab_loss(X[:, :60].contiguous(), W[:, :60].contiguous(), t),
                lambda: m.vocab_loss(X[:0], W, t[:0]),
                lambda: m.vocab_loss(X, W[:0], t),
                lambda: m.flash_mca_vocab_loss(X, W, t, lse, lse, torch.empty(
                    1 << 20, dtype=torch.uint8, device="cuda")),        # loss is lse
                lambda: m.flash_mca_vocab_loss(X, W, t, lse, dloss, torch.empty(
                    16, dtype=torch.uint8, device="cuda"))):            # too small
        with pytest.raises(m.FmcaError):
            bad()


@pytest.mark.parametrize("M", [40, 300, 700])
def test_nan_in_the_vocabulary_leaves_ignored_rows_zero(M):
    m = fm()
    X, W, t, dloss = make(M, 3000, 64, 0.5, 95)
    W[11, 3] = float("nan")
    loss, lse, dX, dW = run(m, X, W, t, dloss)
    out = (t < 0) | (t >= 3000)
    assert (loss[out] == 0).all() and (lse[out] == 0).all() and (dX[out] == 0).all()
    assert torch.isnan(loss[~out]).all() and torch.isnan(dX[~out]).all()


@pytest.mark.parametrize("M", [5000, 100])
def test_shifted_labels(M):
    """The next token's label for each token: target, dloss and lse start where
    only their own type is aligned."""
    m = fm()
    X, W, t, dloss = make(M, 300, 64, 0.7, 97)
    ref = run(m, X, W, t, dloss)
    pad = lambda v: torch.cat([v[:1], v])[1:]  # noqa: E731
    t1, g1, l1 = pad(t), pad(dloss), pad(ref[1])
    assert t1.data_ptr() % 16 == 8 and g1.data_ptr() % 16 == 4
    loss, lse = m.vocab_loss(X, W, t1)
    got = (loss, lse) + m.vocab_loss_backward(X, W, t1, l1, g1)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("keep", [1.0, 0.3])
@pytest.mark.parametrize("M,V,d", [(100, 19456, 64), (100, 19457, 64), (300, 6400, 64),
                                   (300, 6401, 64), (600, 3840, 72), (600, 3841, 72),
                                   (2000, 1150, 64)])
def test_both_sides_of_the_small_tiles(M, V, d, keep):
    """Products go in 128 x 128 tiles while those fit on the CTAs at once."""
    check(fm(), *make(M, V, d, keep, M + V))
