"""One training step of a GAU layer with its norms and loss, all through the
package: norm -> projections -> core -> output projection -> norm with the
residual branch -> vocabulary loss, and back, against the same network in fp64
torch operations differentiated by autograd.

Bound: along a gradient's path the step rounds to bf16 about 22 times (forward:
the norm, the projections, the core's rows, weights and states, its output, the
projection, the sum and its norm; backward the same stages and the loss's
probabilities), each by at most 2^-8 of the value and independently of the
others: sqrt(22) 2^-8 = 1.8e-2 of the gradient's 2-norm; twice that allows for
the stages that stretch an error (the squared relu, the norms).
"""
from __future__ import annotations

import pytest
import torch

import oracle.backward as core_oracle

from tests.test_gpu_parity import fm

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
BOUND = 2 * 22 ** 0.5 * 2.0 ** -8


def parameters(d, e, s, V, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *k, scale=1.0, shift=0.0: scale * torch.randn(*k, generator=g) + shift  # noqa: E731
    return {"w1": n(d, scale=0.1, shift=1.0), "b1": n(d, scale=0.1),
            "Wt": n(2 * e + s, d, scale=1.5 * d ** -0.5).to(BF),
            "gamma": n(4, s, scale=0.1, shift=1.0), "beta": n(4, s, scale=0.1),
            "Wo": n(d, e, scale=4 * e ** -0.5).to(BF),
            "w2": n(d, scale=0.1, shift=1.0), "b2": n(d, scale=0.1),
            "Wv": n(V, d, scale=2 * d ** -0.5).to(BF)}


def step(m, p, x, target, dloss, B, n, C, e, s, causal):
    """(loss, gradients) of the step on the GPU."""
    y1, _, mean1, rstd1 = m.layer_norm(x, p["w1"], p["b1"])
    U, V, Z = m.gau_project(y1, p["Wt"], e, s)
    seq = lambda t: t.view(B, n, -1)  # noqa: E731
    O = m.forward(seq(Z), seq(V), seq(U), p["gamma"], p["beta"], C, causal)
    out = m.gau_output(O.view(B * n, e), p["Wo"])
    y2, h2, mean2, rstd2 = m.layer_norm(out, p["w2"], p["b2"], residual=x)
    loss, lse = m.vocab_loss(y2, p["Wv"], target)

    dy2, dWv = m.vocab_loss_backward(y2, p["Wv"], target, lse, dloss)
    dh2, dw2, db2 = m.layer_norm_backward(dy2, h2, p["w2"], mean2, rstd2)
    dO, dWo = m.gau_output_backward(O.view(B * n, e), p["Wo"], dh2)
    dZ, dV, dU, dgamma, dbeta = m.backward(seq(Z), seq(V), seq(U), p["gamma"], p["beta"], seq(dO),
                                           C, causal)
    rows = lambda t: t.view(B * n, -1)  # noqa: E731
    dy1, dWt = m.gau_project_backward(y1, p["Wt"], rows(dU), rows(dV), rows(dZ))
    dx, dw1, db1 = m.layer_norm_backward(dy1, x, p["w1"], mean1, rstd1, dh=dh2)
    return loss, {"x": dx, "w1": dw1, "b1": db1, "Wt": dWt, "gamma": dgamma, "beta": dbeta,
                  "Wo": dWo, "w2": dw2, "b2": db2, "Wv": dWv}


def reference(p, x, target, dloss, B, n, C, e, s, causal):
    q = {k: v.double().requires_grad_(True) for k, v in {**p, "x": x}.items()}
    F = torch.nn.functional
    d = x.shape[1]
    y1 = F.layer_norm(q["x"], (d,), q["w1"], q["b1"], 1e-5)
    U, V, Z = torch.split(F.silu(y1 @ q["Wt"].T), [e, e, s], 1)
    seq = lambda t: t.reshape(B, n, -1)  # noqa: E731
    O = core_oracle.forward_torch(seq(Z), seq(V), seq(U), q["gamma"], q["beta"], C, causal)
    out = O.reshape(B * n, e) @ q["Wo"].T
    y2 = F.layer_norm(out + q["x"], (d,), q["w2"], q["b2"], 1e-5)
    loss = F.cross_entropy(y2 @ q["Wv"].T, target, ignore_index=-100, reduction="none")
    grads = torch.autograd.grad((loss * dloss.double()).sum(), list(q.values()))
    return loss.detach(), dict(zip(q, grads))


@pytest.mark.parametrize("causal,keep", [(True, 1.0), (False, 0.15)], ids=["causal", "masked"])
def test_training_step(causal, keep):
    m = fm()
    B, n, C, d, e, s, V = 2, 512, 256, 192, 256, 128, 1000
    p = parameters(d, e, s, V, 3)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B * n, d, generator=g).to(BF)
    target = torch.randint(0, V, (B * n,), generator=g)
    target[torch.rand(B * n, generator=g) >= keep] = -100
    dloss = torch.full((B * n,), 1.0 / int((target >= 0).sum()))
    args = (B, n, C, e, s, causal)
    loss, grads = step(m, {k: v.cuda() for k, v in p.items()}, x.cuda(), target.cuda(),
                       dloss.cuda(), *args)
    torch.cuda.synchronize()
    assert m.flash_mca_device_status()[0] == m.FMCA_OK
    rloss, rgrads = reference(p, x, target, dloss, *args)

    def off(a, r):
        a = a.double().cpu()
        return float((a - r).norm() / r.norm())
    assert off(loss, rloss) <= BOUND
    for name, ref in rgrads.items():
        assert off(grads[name], ref) <= BOUND, f"{name}: {off(grads[name], ref):.3e}"


def test_captured_step_follows_its_inputs():
    """The whole step as one graph, replayed on new tokens and targets."""
    m = fm()
    B, n, C, d, e, s, V = 1, 512, 256, 192, 256, 128, 500
    p = {k: v.cuda() for k, v in parameters(d, e, s, V, 5).items()}
    g = torch.Generator().manual_seed(6)
    feeds = []
    for keep in (1.0, 0.2, 0.6):
        t = torch.randint(0, V, (n,), generator=g)
        t[torch.rand(n, generator=g) >= keep] = -100
        feeds.append((torch.randn(n, d, generator=g).to(BF).cuda(), t.cuda(),
                      torch.rand(n, generator=g).cuda()))
    args = (B, n, C, e, s, True)
    want = [step(m, p, *f, *args) for f in feeds]
    x, t, w = [v.clone() for v in feeds[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grads = step(m, p, x, t, w, *args)
    for f, (rloss, rgrads) in zip(feeds, want):
        for dst, src in zip((x, t, w), f):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, rloss)
        for k in grads:
            assert torch.equal(grads[k], rgrads[k]), k
