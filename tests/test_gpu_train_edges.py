"""The training operators where few calls go: rows taken as they are over several
pieces of the vocabulary, arrays past 2^31 bytes and elements, calls behind the
kernel or copy that writes one of their operands, and the loss's gradients
against differences along a direction, with independent roundings in quadrature.
"""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_parity import fm
from tests.test_gpu_vocab_loss import R, check, make, reference, run

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# ------------------------------------------- few rows, a vocabulary in pieces

@pytest.mark.parametrize("keep", [1.0, 0.3])
@pytest.mark.parametrize("M,V,d", [(100, 530000, 8), (100, 530000, 64), (300, 263000, 8)])
def test_rows_as_they_are_over_pieces(M, V, d, keep):
    check(fm(), *make(M, V, d, keep, M + V + d))


@pytest.mark.parametrize("M,V,d", [(100, 530000, 64), (300, 263000, 8)])
def test_ignored_rows_reach_nothing_over_pieces(M, V, d):
    m = fm()
    X, W, t, dloss = make(M, V, d, 0.5, 5)
    clean = run(m, X, W, t, dloss)
    out = (t < 0) | (t >= V)
    X2, g2 = X.clone(), dloss.clone()
    X2[out], g2[out] = float("nan"), float("inf")
    dirty = run(m, X2, W, t, g2)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
    assert (dirty[2][out] == 0).all()


# ------------------------------------------------------------ tall arrays
# Only the last rows hold anything; what the call leaves there is compared with a
# call on those rows alone.

TAIL = 200


def tall(M, tail):
    t = torch.zeros((M,) + tail.shape[1:], dtype=tail.dtype, device="cuda")
    t[-len(tail):] = tail
    return t


@pytest.mark.parametrize("d,dt", [(1024, BF), (1023, BF), (1022, BF), (1021, torch.float32)],
                         ids=lambda v: str(v).removeprefix("torch."))
def test_layer_norm_backward_past_32_bits(d, dt):
    m = fm()
    M = (1 << 31) // d + 300
    g = torch.Generator(device="cuda").manual_seed(d)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    dy, h, dh = [n(TAIL, d).to(dt) for _ in range(3)]
    w, mean, rstd = 1 + 0.2 * n(d), 0.1 * n(TAIL), 1 + 0.1 * n(TAIL)
    want = m.layer_norm_backward(dy, h, w, mean, rstd, dh)
    dx, dw, db = m.layer_norm_backward(tall(M, dy), tall(M, h), w, tall(M, mean), tall(M, rstd),
                                       tall(M, dh))
    assert torch.equal(dx[-TAIL:], want[0]) and not dx[:1000].any() and not dx[-1200:-TAIL].any()
    # the same 200 terms in another order, and zeros: 200 + 40 roundings of partial
    # sums at most
    xhat = (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for a, b, terms in ((dw, want[1], dy.double() * xhat), (db, want[2], dy.double())):
        assert ((a.double() - b.double()).abs() <= 480 * 2.0 ** -24 * terms.abs().sum(0)).all()


def test_projection_gradients_up_to_32_bits():
    """The tallest batch of 192 columns that is accepted, and one row more."""
    m = fm()
    d, e, s = 64, 64, 64
    M = ((1 << 31) - 1) // 192
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *k: torch.randn(*k, device="cuda", generator=g).to(BF)  # noqa: E731
    X, Wt, up = n(TAIL, d), (n(192, d).float() / 8).to(BF), [n(TAIL, 64) for _ in range(3)]
    dX, dWt = m.gau_project_backward(tall(M, X), Wt, *[tall(M, u) for u in up])
    want = m.gau_project_backward(X, Wt, *up)
    # rows of dX: three k steps, in the same order in either call
    assert torch.equal(dX[-TAIL:], want[0]) and not dX[:1000].any() and not dX[-1200:-TAIL].any()
    # dWt: the tail's terms in another order (fp32 sums of 200 products), each side
    # rounded once
    x = X.double()
    pre = x @ Wt.double().T
    sig = torch.sigmoid(pre)
    dpre = (torch.cat(up, 1).double() * sig * (1 + pre * (1 - sig))).abs()
    assert ((dWt.double() - want[1].double()).abs()
            <= 2 * R * want[1].double().abs() + 400 * 2.0 ** -23 * (dpre.T @ x.abs())).all()
    with pytest.raises(m.FmcaError):
        m.gau_project_backward(tall(M + 1, X), Wt, *[tall(M + 1, u) for u in up])


def test_output_gradients_up_to_32_bits():
    m = fm()
    e, d = 64, 64
    M = (1 << 25) - 1
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *k: torch.randn(*k, device="cuda", generator=g).to(BF)  # noqa: E731
    Y, Wo, dOut = n(TAIL, e), n(d, e), n(TAIL, d)
    dY, dWo = m.gau_output_backward(tall(M, Y), Wo, tall(M, dOut))
    want = m.gau_output_backward(Y, Wo, dOut)
    assert torch.equal(dY[-TAIL:], want[0]) and not dY[:1000].any() and not dY[-1200:-TAIL].any()
    assert ((dWo.double() - want[1].double()).abs() <= 2 * R * want[1].double().abs()
            + 400 * 2.0 ** -23 * (dOut.double().abs().T @ Y.double().abs())).all()
    with pytest.raises(m.FmcaError):
        m.gau_output_backward(tall(M + 1, Y), Wo, tall(M + 1, dOut))


@pytest.mark.parametrize("every", [False, True], ids=["tail", "every row"])
def test_vocab_loss_up_to_32_bits(every):
    """33.5 million rows against 300 entries (two pieces); a target at the last rows
    or at all of them, whose X is 0 elsewhere: loss log 300, nothing for dW."""
    m = fm()
    V, d = 300, 64
    M = (1 << 25) - 1
    X, W, t, dloss = make(TAIL, V, d, 1.0, 3)
    target = torch.full((M,), 7 if every else -100, device="cuda")
    target[-TAIL:] = t
    Xt, gt = tall(M, X), torch.full((M,), 0.5, device="cuda")
    gt[-TAIL:] = dloss
    loss, lse, dX, dW = run(m, Xt, W, target, gt)
    torch.cuda.synchronize()
    assert m.flash_mca_device_status()[0] == m.FMCA_OK
    refs = reference(X, W, t, dloss)
    got = (loss[-TAIL:], lse[-TAIL:], dX[-TAIL:], dW)
    for name, a, (ref, bound) in zip(("loss", "lse", "dX", "dW"), got, refs):
        assert ((a.double() - ref).abs() <= bound).all(), name
    if every:
        logv = torch.log(torch.tensor(300.0, dtype=torch.float64)).item()
        assert ((loss[:-TAIL].double() - logv).abs() <= 2.0 ** -20 * (1 + logv)).all()
        # every such row has the gradient 0.5 (mean of W - W[7])
        z = torch.zeros(1, d, device="cuda", dtype=BF)
        ref, bound = reference(z, W, torch.tensor([7], device="cuda"), gt[:1])[2]
        for rows in (dX[:1000], dX[M // 2:M // 2 + 1000], dX[-1200:-TAIL]):
            assert ((rows.double() - ref).abs() <= bound).all()
    else:
        assert not loss[:-TAIL].any() and not dX[:1000].any() and not dX[-1200:-TAIL].any()


# -------------------------------------------- calls behind what writes an operand

CASES = [("norm", "x"), ("norm", "w"), ("norm backward", "dy"), ("norm backward", "mean"),
         ("loss", "X"), ("loss", "W"), ("loss", "target"), ("loss backward", "W"),
         ("loss backward", "dloss"), ("loss backward", "lse"), ("output", "Y"), ("output", "Wo"),
         ("output", "dOut"), ("project", "X"), ("project", "Wt"), ("project", "dV")]


@pytest.mark.parametrize("M", [100, 700])
@pytest.mark.parametrize("op,name", CASES)
def test_calls_behind_the_writer_of_an_operand(op, name, M):
    """An operand is cleared and then written by an elementwise kernel, or by a
    copy, just ahead of the call, captured and not."""
    m = fm()
    g = torch.Generator(device="cuda").manual_seed(M)
    r = lambda *k: (torch.randn(*k, device="cuda", generator=g) / 8).to(BF)  # noqa: E731
    f = lambda *k: torch.randn(*k, device="cuda", generator=g)  # noqa: E731
    a = {"x": r(M, 128), "w": f(128), "b": f(128), "dy": r(M, 128), "mean": f(M) / 8,
         "rstd": 1 + f(M) / 8, "X": r(M, 128), "W": r(900, 128), "dloss": f(M),
         "target": torch.arange(M, device="cuda") % 900, "Y": r(M, 256), "Wo": r(128, 256),
         "dOut": r(M, 128), "Wt": r(576, 128), "dU": r(M, 256), "dV": r(M, 256), "dZ": r(M, 64)}
    a["lse"] = m.vocab_loss(a["X"], a["W"], a["target"])[1]
    call = {
        "norm": lambda: [m.layer_norm(a["x"], a["w"], a["b"])[k] for k in (0, 2, 3)],
        "norm backward": lambda: m.layer_norm_backward(a["dy"], a["x"], a["w"], a["mean"], a["rstd"]),
        "loss": lambda: m.vocab_loss(a["X"], a["W"], a["target"]),
        "loss backward": lambda: m.vocab_loss_backward(a["X"], a["W"], a["target"], a["lse"],
                                                       a["dloss"]),
        "output": lambda: m.gau_output_backward(a["Y"], a["Wo"], a["dOut"]),
        "project": lambda: m.gau_project_backward(a["X"], a["Wt"], a["dU"], a["dV"], a["dZ"]),
    }[op]
    operand, keep = a[name], a[name].clone()
    want = [o.clone() for o in call()]
    operand.zero_()
    assert not all(torch.equal(p, q) for p, q in zip(call(), want))  # the call reads it

    def kernel():
        operand.zero_()
        torch.mul(keep, 1, out=operand)
        return call()

    def copy():
        operand.zero_()
        operand.copy_(keep)
        return call()

    for way in (kernel, copy):
        for _ in range(3):
            got = way()
            assert all(torch.equal(p, q) for p, q in zip(got, want))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = way()
        for _ in range(3):
            operand.fill_(3)
            for o in got:
                o.fill_(0)
            graph.replay()
            assert all(torch.equal(p, q) for p, q in zip(got, want))


# ------------------------------------------------------------ differences

@pytest.mark.parametrize("scaled", [1.0, 1.1, 0.9])
def test_gradients_are_differences_along_directions(scaled):
    """The summed loss's change along random directions v and along the gradient
    itself.  A half step of bf16 has a deviation of R / sqrt 3 at most, relative
    to the value: the gradient's entries bring (R^2 / 3) sum (G v)^2 to the slope's
    variance, the entries q of (p - onehot) g, through the product with v's image
    under the other operand, (R^2 / 3) sum (q u)^2; six deviations, and 1e-5 for
    the difference's own error (h^2 / 6 of the third derivative, ~50 at most, and
    2^-52 of the loss over h) and the fp32 sums.  A gradient that is off by a tenth
    along itself is outside."""
    m = fm()
    X, W, t, dloss = make(128, 300, 64, 0.8, 91, scale=1.0)
    _, lse = m.vocab_loss(X, W, t)
    got = m.vocab_loss_backward(X, W, t, lse, dloss)
    x, w = X.double(), W.double()
    has = (t >= 0) & (t < 300)
    weight = torch.where(has, dloss.double(), torch.zeros_like(dloss.double()))
    at = torch.where(has, t, torch.zeros_like(t))

    def total(a, b):
        z = a @ b.T
        return ((torch.logsumexp(z, 1) - z.gather(1, at[:, None])[:, 0]) * weight).sum()
    z = x @ w.T
    q = torch.softmax(z, 1)
    q[torch.arange(128), at] -= 1.0
    q *= weight[:, None]
    refs = (q @ w, q.T @ x)
    g = torch.Generator(device="cuda").manual_seed(1)
    outside = 0
    for which in (0, 1):
        G = refs[which]
        for k in range(5):
            along = k == 4
            v = G / G.norm() if along else torch.randn(G.shape, generator=g, device="cuda",
                                                       dtype=torch.float64)
            h = 1e-4
            ends = [total(*((x + sgn * v, w) if which == 0 else (x, w + sgn * v)))
                    for sgn in (h, -h)]
            slope = float((ends[0] - ends[1]) / (2 * h))
            u = v @ w.T if which == 0 else x @ v.T  # [M][V]
            bound = 6 * (R ** 2 / 3 * (((G * v) ** 2).sum() + ((q * u) ** 2).sum())).sqrt() + 1e-5
            off = abs(slope - scaled * float((got[which].double() * v).sum()))
            if scaled == 1.0:
                assert off <= bound
            elif along:
                outside += off > bound
    assert scaled == 1.0 or outside == 2


# ------------------------------------------------------- several calls at once

def small_step(m, M, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *k: (torch.randn(*k, device="cuda", generator=g) / 8).to(BF)  # noqa: E731
    X, W, Y, Wo, dOut = r(M, 136), r(1500, 136), r(M, 264), r(128, 264), r(M, 128)
    Wt, dU, dV, dZ = r(2 * 256 + 64, 136), r(M, 256), r(M, 256), r(M, 64)
    t = torch.randint(-200, 1500, (M,), device="cuda", generator=g)
    w, dl = torch.rand(136, device="cuda", generator=g), torch.rand(M, device="cuda", generator=g)

    def step():
        y, h, mean, rstd = m.layer_norm(X, w, w)
        loss, lse = m.vocab_loss(y, W, t)
        dX, dW = m.vocab_loss_backward(y, W, t, lse, dl)
        return (y, loss, dX, dW, *m.layer_norm_backward(dX, h, w, mean, rstd),
                *m.gau_output_backward(Y, Wo, dOut), *m.gau_project_backward(X, Wt, dU, dV, dZ))
    return step


def test_threads_with_a_stream_each():
    import threading
    m = fm()
    steps = [small_step(m, M, M) for M in (90, 700, 1300)]
    want = [[o.clone() for o in s()] for s in steps]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = steps[k]()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    wrong.append(k)
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and m.flash_mca_device_status()[0] == m.FMCA_OK


def test_graphs_replayed_side_by_side():
    m = fm()
    steps = [small_step(m, M, M) for M in (90, 700, 1300)]
    want = [[o.clone() for o in s()] for s in steps]
    torch.cuda.synchronize()
    graphs = []
    for s in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s()
        graphs.append((graph, out, torch.cuda.Stream()))
    for _ in range(20):
        for graph, _, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out, _), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert m.flash_mca_device_status()[0] == m.FMCA_OK


def test_a_single_row_without_leading_dimensions():
    m = fm()
    x, w = torch.randn(301, device="cuda"), torch.rand(301, device="cuda")
    y, h, mean, rstd = m.layer_norm(x, w, w, residual=x)
    y2, h2, mean2, rstd2 = m.layer_norm(x[None], w, w, residual=x[None])
    assert mean.shape == () and torch.equal(y, y2[0]) and torch.equal(h, 2 * x)
    got = m.layer_norm_backward(x, h, w, mean, rstd, x)
    want = m.layer_norm_backward(x[None], h2, w, mean2, rstd2, x[None])
    assert torch.equal(got[0], want[0][0]) and all(torch.equal(a, b) for a, b in
                                                  zip(got[1:], want[1:]))
