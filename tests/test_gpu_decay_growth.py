"""Linear attention with log decays above 0: a state that grows, up to and past the range of
32 bits.

Bounds as in the tests of the decays below 0: sums of absolute values (oracle.serve) times
the number of roundings that a term goes through, 2^-23 each, and for bf16 half a step
(2^-8) for the output, the weights and the state as an operand.  Token by token a term is
multiplied and rounded at most T times."""
import math

import numpy as np
import pytest
import torch

import flash_mixed_chunk_gb300 as fm
from oracle import serve

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# what the tensor cores take, what they do not, and 32 bits
FORMS = [(BF16, 64, 64), (BF16, 128, 72), (BF16, 20, 70), (F32, 64, 64), (F32, 9, 130)]


def make(B, T, H, dk, dv, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    q, k, v = (torch.randn(B, T, H, d, generator=g).to(dtype).cuda() for d in (dk, dk, dv))
    return q, k, v, torch.randn(B, H, dk, dv, generator=g).cuda()


def check(o, s, want, dk, T, dtype):
    """Of the values that fit 32 bits with room for partial sums."""
    ro, rs, sz = want
    tol = (2 * dk + 2 * T + 64) * 2.0 ** -23 * sz["whole"]
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -16) * (sz["near"] + sz["far"])
    got, fits = o.float().cpu().numpy(), sz["whole"] < 1e37
    assert (np.abs(got[fits] - ro[fits]) <= tol[fits]).all()
    got, fits = s.cpu().numpy(), sz["state"] < 1e37
    assert (np.abs(got[fits] - rs[fits]) <= (3 * T + 64) * 2.0 ** -23 * sz["state"][fits]).all()


def settled():
    torch.cuda.synchronize()
    assert fm.flash_mca_device_status()[0] == fm.FMCA_OK


def test_a_step_whose_decay_leaves_the_range():
    """exp(log_decay) is an infinity in 32 bits: the state one of its signs."""
    H = 33
    q, k, v, state = make(3, 1, H, 8, 8, F32)
    ld = torch.linspace(88.8, 120.0, H).cuda()
    ld[-2], ld[-1] = math.inf, 0.5
    before = state.clone()
    fm.decay_step(q[:, 0], k[:, 0], v[:, 0], ld, state)
    settled()
    assert torch.equal(state[:, :-1], before[:, :-1] * math.inf)
    assert torch.isfinite(state[:, -1]).all()


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
@pytest.mark.parametrize("T,rate", [(1, 3.0), (5, 1.0), (100, 0.05), (130, 0.3), (130, 0.35),
                                    (300, 1e-4), (300, 0.14), (300, 0.2), (300, 0.245),
                                    (1500, 0.03)])
def test_growth_within_the_range(T, rate, dtype, dk, dv):
    q, k, v, state = make(2, T, 3, dk, dv, dtype)
    ld = torch.tensor([rate, -rate, rate / 7]).cuda()
    lengths = torch.tensor([T, T // 2], dtype=torch.int32).cuda()
    for s0, n in ((None, None), (state, None), (state, lengths)):
        o, s = fm.decay_attention(q, k, v, ld, state=s0, scale=0.3, lengths=n)
        settled()
        want = serve.decay_attention(q, k, v, ld, s0, 0.3, n)
        assert (want[2]["whole"] < 1e37).all()
        check(o, s, want, dk, T, dtype)


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
def test_what_is_zero_stays_zero(dtype, dk, dv):
    """A power outside the range that meets a state or a key of zero: the formula is finite
    there."""
    q, k, v, _ = make(1, 400, 3, dk, dv, dtype)
    k[:, :390] = 0
    ld = torch.tensor([1.0, 0.7, 0.24]).cuda()
    o, s = fm.decay_attention(q, k, v, ld)
    settled()
    want = serve.decay_attention(q, k, v, ld)
    assert (want[2]["whole"] < 1e37).all()
    check(o, s, want, dk, 400, dtype)
    assert not o[:, :390].any()
    q, k, v, _ = make(1, 100, 3, dk, dv, dtype)
    k[:, :90] = 0
    o, s = fm.decay_attention(q, k, v, ld)
    settled()
    check(o, s, serve.decay_attention(q, k, v, ld), dk, 100, dtype)
    state = torch.zeros(1, 3, dk, dv, device="cuda")
    state[0, 1, 0, 0] = 2.0 ** -100  # grows by 2^216, and fits all the same
    k.zero_()
    o, s = fm.decay_attention(q, k, v, torch.full((3,), 1.5).cuda(), state=state)
    settled()
    want = serve.decay_attention(q, k, v, [1.5] * 3, state)
    check(o, s, want, dk, 100, dtype)
    assert s[0, 1, 0, 0] > 1e34


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
@pytest.mark.parametrize("T", [130, 1500])
def test_past_the_range_comes_the_infinity(T, dtype, dk, dv):
    """Positive operands: rows up to the overflow as the formula has them, then +inf, and a
    head that does not grow as without the others."""
    q, k, v, state = (x.abs() + 0.1 for x in make(1, T, 2, dk, dv, dtype))
    ld = torch.tensor([1.2, -0.1]).cuda()
    o, s = fm.decay_attention(q, k, v, ld, state=state)
    settled()
    with np.errstate(over="ignore"):
        want = serve.decay_attention(q, k, v, ld, state)
    check(o, s, want, dk, T, dtype)
    big = torch.as_tensor(want[0] > 1e39)
    assert big.any() and torch.isposinf(o.cpu()[big]).all()
    assert torch.isposinf(s[0, 0]).all()
    p, t = fm.decay_attention(q[:, :, 1:], k[:, :, 1:], v[:, :, 1:], ld[1:], state=state[:, 1:])
    settled()
    tol = 2.0 ** -7 if dtype == BF16 else (3 * T + 64) * 2.0 ** -22
    assert ((o[:, :, 1:] - p).abs() <= tol * p.abs()).all()
    assert ((s[:, 1:] - t).abs() <= (3 * T + 64) * 2.0 ** -22 * t.abs()).all()


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
def test_growing_heads_in_place_behind_their_end_and_in_pieces(dtype, dk, dv):
    T = 2500  # cut into segments
    q, k, v, state = make(2, T, 1, dk, dv, dtype)
    ld = torch.tensor([0.03]).cuda()
    lengths = torch.tensor([T, 1600], dtype=torch.int32).cuda()
    k[:, :T - 1000] *= 2.0 ** -60
    state *= 2.0 ** -90
    o = torch.full((2, T, 1, dv), 7.0, dtype=dtype, device="cuda")
    need = fm.flash_mca_decay_workspace_bytes(q, k, v, ld)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    place = state.clone()
    fm.flash_mca_decay_attention(q, k, v, ld, lengths, place, o, place, ws)
    p, t = fm.decay_attention(q, k, v, ld, state=state, lengths=lengths)
    settled()
    assert torch.equal(place, t) and torch.equal(o, p) and not o[1, 1600:].any()
    want = serve.decay_attention(q, k, v, ld, state, 1.0, lengths)
    assert (want[2]["whole"] < 1e37).all()
    check(p, t, want, dk, T, dtype)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        po, pt = fm.decay_attention(q, k, v, ld, state=state, lengths=lengths)
    graph.replay()
    settled()
    assert torch.equal(po, p) and torch.equal(pt, t)
