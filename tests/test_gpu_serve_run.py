"""Generation with states as it is used: prompts, then beam search over single tokens with
the states, the core's own decode state and the histories following the parents, eager and
as a captured step."""
import math

import numpy as np
import pytest
import torch

import flash_mixed_chunk_gb300 as fm
from oracle import serve

pytestmark = pytest.mark.gpu

B, K, H, DK, DV, V, E = 2, 4, 2, 16, 32, 128, 64


def model(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"emb": r(V, E), "qkv": r(E, H * (2 * DK + DV)) / math.sqrt(E),
            "out": r(V, H * DV) / math.sqrt(H * DV) * 3,
            "ld": torch.tensor([-0.05, -0.4])}


def split(x):
    q, k, v = x.split([H * DK, H * DK, H * DV], -1)
    return q.unflatten(-1, (H, DK)), k.unflatten(-1, (H, DK)), v.unflatten(-1, (H, DV))


def test_a_search_against_the_oracle():
    m = model()
    dev = {k: v.cuda() for k, v in m.items()}
    g = torch.Generator().manual_seed(9)
    T, steps = 150, 6
    prompt = torch.randint(0, V, (B, T), generator=g)
    lengths = torch.tensor([150, 97], dtype=torch.int32)

    # the framework, in 32 bits
    q, k, v = split(dev["emb"][prompt.cuda()] @ dev["qkv"])
    _, state = fm.decay_attention(q, k, v, dev["ld"], lengths=lengths.cuda())
    state = state.repeat_interleave(K, 0)
    scores = torch.tensor([[0.0] + [-math.inf] * (K - 1)] * B).cuda()
    history = torch.zeros(B, K, steps, dtype=torch.int64, device="cuda")
    finished = torch.zeros(B, K, dtype=torch.bool, device="cuda")
    last = prompt[torch.arange(B), lengths.long() - 1].cuda()[:, None].repeat(1, K)
    for t in range(steps):
        q, k, v = split(dev["emb"][last.flatten()] @ dev["qkv"])
        o = fm.decay_step(q, k, v, dev["ld"], state)
        logits = o.flatten(1) @ dev["out"].T
        scores, parent, last = fm.beam_select(logits, scores, finished=finished, pad=0)
        fm.beam_reorder([state, history, finished], parent)
        history[:, :, t] = last
        finished |= last == 1
    torch.cuda.synchronize()

    # the same in 64 bits with the oracle's steps
    d = {k: v.double().numpy() for k, v in m.items()}
    cut = [H * DK, 2 * H * DK]

    def parts(x):
        a, b, c = np.split(x, cut, axis=-1)
        return (a.reshape(*a.shape[:-1], H, DK), b.reshape(*b.shape[:-1], H, DK),
                c.reshape(*c.shape[:-1], H, DV))

    _, st, _ = serve.decay_attention(*parts(d["emb"][prompt.numpy()] @ d["qkv"]), d["ld"], None,
                                     1.0, lengths)
    st = np.repeat(st, K, 0)
    sc = np.array([[0.0] + [-np.inf] * (K - 1)] * B)
    hist, fin = np.zeros((B, K, steps), np.int64), np.zeros((B, K), bool)
    last = np.repeat(prompt.numpy()[np.arange(B), lengths.numpy() - 1][:, None], K, 1)
    for t in range(steps):
        x = parts(d["emb"][last.ravel()] @ d["qkv"])
        o, st, _ = serve.decay_attention(*[y[:, None] for y in x], d["ld"], st)
        sc, par, last = serve.beam_select(o.reshape(B, K, -1) @ d["out"].T, sc, K, fin)
        st = serve.reorder(st, par)
        hist = serve.reorder(hist.reshape(B * K, -1), par).reshape(B, K, steps)
        fin = serve.reorder(fin.reshape(B * K, 1), par).reshape(B, K)
        hist[:, :, t] = last
        fin |= last == 1
    assert history.cpu().numpy().tolist() == hist.tolist()
    assert np.allclose(scores.cpu().numpy(), sc, rtol=1e-5, atol=1e-4)
    assert np.allclose(state.cpu().numpy(), st, rtol=1e-3, atol=1e-3)


def test_a_captured_step_is_the_eager_one():
    """One decoding step with projections, the core's decode step, the decay step, logits,
    selection and reordering, replayed, against the same calls one by one."""
    g = torch.Generator().manual_seed(3)
    n, s, e, C, t, code = B * K, 64, 64, 16, 5, fm.FMCA_BF16
    bf = torch.bfloat16
    r = lambda *x: torch.randn(*x, generator=g).cuda()  # noqa: E731
    Wt, Wv, x0 = r(2 * e + s, E).mul_(0.1).to(bf), r(V, e).to(bf), r(V, E).to(bf)
    gamma, beta, ld = r(4, s), r(4, s), torch.tensor([-0.1, -0.5]).cuda()
    core0 = torch.zeros(fm.flash_mca_decode_state_bytes(n, s, e, C, code), dtype=torch.uint8,
                        device="cuda")
    state0 = r(n, H, 32, 32)

    def fresh():
        return {"core": core0.clone(), "state": state0.clone(),
                "scores": -torch.arange(n, device="cuda").view(B, K).float() / 7,
                "last": torch.arange(n, device="cuda").view(B, K) % V,
                "history": torch.zeros(B, K, 8, dtype=torch.int64, device="cuda")}

    o = torch.empty(n, e, dtype=bf, device="cuda")

    def step(c):
        u, v, z = fm.gau_project(x0[c["last"].flatten()], Wt, e, s)
        fm.flash_mca_decode_step(z, v, u, gamma, beta, o, C, t, c["core"], n_norm=64)
        q = o.view(n, 2, 32)
        y = fm.decay_step(q, q, v.view(n, 2, 32), ld, c["state"], scale=0.2)
        logits = fm.gau_output(y.view(n, 64), Wv)
        score, parent, token = fm.beam_select(logits, c["scores"])
        fm.beam_reorder([c["state"], c["history"]], parent)
        fm.flash_mca_decode_reorder(c["core"], parent, s, e, C, t + 1, code)
        c["scores"].copy_(score)
        c["last"].copy_(token)
        c["history"][:, :, 0] = token

    a, b = fresh(), fresh()
    for _ in range(3):
        step(a)
    warm = fresh()
    step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for key, x in fresh().items():
        b[key].copy_(x)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert fm.flash_mca_device_status()[0] == fm.FMCA_OK
    for key in ("scores", "last", "history", "state"):
        assert torch.equal(a[key], b[key]), key
