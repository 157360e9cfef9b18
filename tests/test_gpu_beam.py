"""Beam search's selection and the reordering of rows on the GPU against the oracle.

Parents and tokens have to be the oracle's: the inputs keep candidates of different
beams 1e-5 apart, or exactly equal.  A score is one rounding (half a step, 2^-24) from
a value whose lse is within 1e-6 of the exact one."""
import math

import numpy as np
import pytest
import torch

import flash_mixed_chunk_gb300 as fm
from oracle import serve

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def apart(logits, scores, n, finished):
    """Whether the oracle's first n + 1 candidates of each element differ by 1e-5 or are
    of one beam (or equal, in rows that are)."""
    best, parent, _ = serve.beam_select(logits, scores, n + 1, finished)
    gap = best[:, :-1] - best[:, 1:]
    with np.errstate(invalid="ignore"):
        return ((gap > 1e-5) | (parent[:, :-1] == parent[:, 1:]) | ~np.isfinite(gap)).all()


def check(logits, scores, n, finished=None, pad=0):
    score, parent, token = fm.beam_select(logits, scores, n, finished, pad)
    torch.cuda.synchronize()
    rs, rp, rt = serve.beam_select(logits, scores, n, finished, pad)
    assert parent.tolist() == rp.tolist() and token.tolist() == rt.tolist()
    s = score.double().cpu().numpy()
    none = np.isneginf(rs)
    assert (np.isneginf(s) == none).all()
    s, rs = s[~none], rs[~none]
    assert (np.abs(s - rs) <= 2.0 ** -24 * np.abs(rs) + 1e-6).all()


def make(B, K, V, dtype, seed=0, scale=2.0):
    g = torch.Generator().manual_seed(seed * 100 + V)
    logits = (torch.randn(B, K, V, generator=g) * scale).to(dtype).cuda()
    scores = (-torch.rand(B, K, generator=g) * 4).cuda()
    return logits, scores


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,K,V,n", [
    (1, 1, 1, 1), (2, 1, 5, 1), (1, 4, 31, 4), (3, 2, 1000, 4), (1, 4, 1024, 8),
    (2, 3, 1025, 6), (5, 4, 2049, 4), (1, 4, 32000, 4), (2, 8, 8191, 16), (1, 16, 5003, 32),
    (1, 32, 777, 32), (70, 2, 3001, 2), (1, 1, 100001, 32), (2, 5, 40002, 10),
])
def test_selection(B, K, V, n, dtype):
    for seed in range(50):
        logits, scores = make(B, K, V, dtype, seed)
        if apart(logits, scores, n, None):
            break
    else:
        pytest.fail("no inputs whose candidates are apart")
    check(logits, scores, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [17, 4000, 9001])
def test_ties_go_to_the_lowest_index(V, dtype):
    B, K = 3, 4
    flat = torch.zeros(B, K, V, dtype=dtype, device="cuda")
    scores = torch.zeros(B, K, device="cuda")
    for n in (1, 8, 32):
        check(flat, scores, n)  # all equal: beam 0's first tokens
    g = torch.Generator().manual_seed(V)
    one = (torch.randn(1, 1, V, generator=g) * 2).round().to(dtype).cuda()
    check(one.expand(B, K, V).contiguous(), scores, 32)  # equal beams, few values
    zeros = flat.clone()
    zeros[:, :, V // 2:] = -0.0
    check(zeros, scores, 8)  # -0 equals 0
    up = torch.arange(V, dtype=F32, device="cuda").div_(V).to(dtype).expand(B, K, V).contiguous()
    check(up, torch.tensor([[0.0, -1.0, -2.0, -3.0]], device="cuda").repeat(B, 1), 20)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 5000, 5001])
def test_masked_and_broken_rows(V, dtype):
    logits, scores = make(4, 5, V, dtype, 3)
    logits[0, :, 7:] = -math.inf          # few tokens allowed
    logits[1, 0] = -math.inf              # nothing allowed
    logits[1, 1, V // 2] = math.nan
    logits[1, 2, V - 1] = math.inf
    logits[1, 3, :-1] = -math.inf         # one token allowed
    logits[2, :, ::2] = torch.finfo(dtype).min
    logits[3] = -math.inf                 # no candidate anywhere
    scores[0, 2:] = -math.inf             # the beams that have not begun
    scores[2, 1], scores[2, 2] = math.nan, math.inf
    for n in (1, 10, 32):
        check(logits, scores, n, pad=3)
    finished = torch.zeros(4, 5, dtype=torch.bool, device="cuda")
    finished[0, 2] = finished[1, 1] = finished[2, 3] = finished[3, 0] = finished[3, 4] = True
    for n in (1, 10, 32):
        check(logits, scores, n, finished, pad=V - 1)
    check(logits, scores, 10, torch.ones_like(finished), pad=0)


def test_far_values_and_sharp_rows():
    logits, scores = make(2, 3, 3000, F32, 1)
    logits[0] *= 1e30
    logits[1, :, 100] = 60.0              # one token has all the weight
    logits[1, 1] -= 1e4
    scores -= 1e3
    assert apart(logits, scores, 4, None)
    check(logits, scores, 4)


def test_rows_apart_and_views():
    B, K, V = 3, 4, 1000
    logits, scores = make(B, K, 1100, BF16, 2)
    wide = logits[:, :, :V]               # a padded vocabulary
    n = 8
    assert apart(wide, scores, n, None)
    check(wide, scores, n)
    check(logits[:, :, 3:V + 3], scores, 4)
    check(wide.reshape(B * K, V), scores, 4)
    for bad in (logits.transpose(1, 2), logits[:, ::2], logits[:2]):
        with pytest.raises(ValueError):
            fm.beam_select(bad, scores)
    for kw, err in ((dict(n=33), fm.FmcaError), (dict(n=0), ValueError), (dict(pad=-1), ValueError),
                    (dict(pad=1100), fm.FmcaError),
                    (dict(finished=torch.zeros(B, K, device="cuda")), ValueError)):
        with pytest.raises(err):
            fm.beam_select(logits, scores, **kw)
    with pytest.raises(TypeError):
        fm.beam_select(logits.half(), scores)
    score = torch.empty(B, 5, device="cuda")
    parent, token = (torch.empty(B, 5, dtype=torch.int64, device="cuda") for _ in range(2))
    fm.flash_mca_beam_select(logits, scores, None, score, parent, token)
    assert torch.equal(torch.stack([parent, token]),
                       torch.stack(fm.beam_select(logits, scores, 5)[1:]))


# ------------------------------------------------------------------- reordering

def reordered(tensors, parent):
    B, K = parent.shape
    rows = [t.reshape(B * K, -1).cpu().view(torch.uint8).numpy() if t.numel() else None
            for t in tensors]
    return [None if r is None else serve.reorder(r, parent.tolist()) for r in rows]


def same(tensors, want):
    for t, w in zip(tensors, want):
        if w is not None:
            n = w.shape[0]
            assert (t.reshape(n, -1).cpu().view(torch.uint8).numpy() == w).all()


@pytest.mark.parametrize("B,K", [(1, 1), (1, 4), (3, 5), (2, 8), (1, 13), (2, 32), (40, 3)])
def test_rows_follow_their_parents(B, K):
    g = torch.Generator().manual_seed(K)
    n = B * K

    def rand(*s):
        return torch.randint(0, 255, s, generator=g, dtype=torch.uint8).cuda()

    base = rand(n * 64 + 1)
    tensors = [rand(n, 5000).view(torch.float32), rand(n, 3, 7), rand(B, K, 6, 16).view(F32),
               rand(n), rand(n, 40).view(torch.int64), base[1:].view(n, 64), rand(n, 0),
               rand(B, K, 12).view(torch.int32)]
    for trial in range(3):
        parent = torch.randint(0, K, (B, K), generator=g).cuda()
        if trial == 1:
            parent = torch.arange(K).expand(B, K).contiguous().cuda()
        if trial == 2 and K > 1:  # a cycle, and parents that are none
            parent = ((torch.arange(K) + 1) % K).expand(B, K).contiguous().cuda()
            parent[0, 0], parent[-1, 1] = -1, K
        want = reordered(tensors, parent)
        (fm.beam_reorder if trial else fm.flash_mca_beam_reorder)(tensors, parent)
        torch.cuda.synchronize()
        same(tensors, want)


def test_rows_of_a_longer_buffer_and_many_tensors():
    B, K = 2, 6
    buf = torch.arange(12 * 50, device="cuda").view(12, 50).clone()
    parent = torch.tensor([[1, 0, 2, 2, 5, 0], [3, 3, 3, 3, 3, 3]], device="cuda")
    want = buf.clone()
    want[:, :20] = torch.as_tensor(serve.reorder(buf[:, :20].cpu(), parent.tolist())).cuda()
    fm.beam_reorder([buf[:, :20]], parent)  # a history so far
    assert torch.equal(buf, want)
    many = [torch.randn(12, 10 + i, device="cuda") for i in range(37)]
    want = reordered(many, parent)
    fm.beam_reorder(many, parent)
    torch.cuda.synchronize()
    same(many, want)
    for bad in ([buf.t()], [buf[:, ::2]], [buf[:11]], [], [buf.cpu()], buf[0, 0]):
        with pytest.raises((ValueError, TypeError)):
            fm.beam_reorder(bad, parent)
    for bad in ([buf, buf], [buf, buf[:, 3:4]]):
        with pytest.raises(fm.FmcaError):
            fm.beam_reorder(bad, parent)
    with pytest.raises(ValueError):
        fm.beam_reorder([buf], parent.int())
    with pytest.raises(fm.FmcaError):
        fm.beam_reorder([torch.zeros(33, 2, device="cuda")],
                        torch.zeros(1, 33, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t", [0, 5, 16, 30])
def test_the_core_decodes_on_from_its_parents(t, dtype):
    """decode_step of reordered beams: what decoding the parents' tokens from the start
    gives, to the bit."""
    B, K, s, e, C = 2, 3, 24, 40, 16
    n = B * K
    code = fm.FMCA_BF16 if dtype == BF16 else fm.FMCA_F32
    g = torch.Generator().manual_seed(t)
    z, v, u = (torch.randn(40, n, d, generator=g).to(dtype).cuda() for d in (s, e, e))
    gamma, beta = (torch.randn(4, s, generator=g).cuda() for _ in range(2))
    parent = torch.tensor([[2, 0, 0], [1, 1, 2]], device="cuda")
    rows = (parent + K * torch.arange(B, device="cuda")[:, None]).flatten()

    def fresh():
        st = torch.zeros(fm.flash_mca_decode_state_bytes(n, s, e, C, code), dtype=torch.uint8,
                         device="cuda")
        fm.flash_mca_decode_reset(st, n, s, e, C, code)
        return st

    def run(st, a, b, order):
        o = torch.empty(b - a, n, e, dtype=dtype, device="cuda")
        for i in range(a, b):
            x = [y[i] if order is None else y[i][order].contiguous() for y in (z, v, u)]
            fm.flash_mca_decode_step(*x, gamma, beta, o[i - a], C, i, st, n_norm=64)
        return o

    a = fresh()
    run(a, 0, t, None)
    fm.flash_mca_decode_reorder(a, parent, s, e, C, t, code)
    got = run(a, t, t + 10, None)
    b = fresh()
    run(b, 0, t, rows)
    assert torch.equal(got, run(b, t, t + 10, None))
