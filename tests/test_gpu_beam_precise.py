"""The logarithm in beam search's selection against 64 bits, where its sum is hard to form:
rows that are nearly flat, whose terms round alike, rows whose maximum comes late, and
candidates of two beams that are closer together than 32 bits tell.

Within u = 2^-24: a term is a difference (u of it), a product with log2 e (u, and 0.22 for the
constant) and ex2.approx (4 u).  What it is a difference from lies up to 2 under the maximum and
moves by more than 2 at a time, with a factor of 5 u each; by their shares of the sum the logits
lie at most ln V under the maximum on average.  A task's terms are a tree of five levels, the
tasks' sums two floats, lanes a tree of five, warps and blocks trees of three with a factor each.
Together under (54 + 5 ln V) u, which a score may be off by.  Candidates of two beams that are
closer than twice as much are decided by sums to 2^-29."""
import math

import numpy as np
import pytest
import torch

import flash_mixed_chunk_gb300 as fm
from oracle import serve

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
FINE = 2.0 ** -29


def bound(V):
    return (54 + 5 * math.log(V)) * 2.0 ** -24


def far(row):
    """max - lse of a row, in 64 bits."""
    z = row.double().cpu()
    return float(z.max() - torch.logsumexp(z, 0))


def first_best(z):
    """Index of each row's largest value, of equal ones the first."""
    return np.argmax(z.float().cpu().numpy(), -1).tolist()


def rows(V, dtype):
    flat = torch.full((V,), -3.7)
    g = torch.Generator().manual_seed(V)
    out = [flat.clone()]
    for p in (0.3, 1.0, 2.5, 4.1, 7.0, 9.3, 12.0):
        for at in (0, V // 2, V - 1):
            x = flat.clone()
            x[at] += p
            out.append(x)
            x = torch.zeros(V)
            x[at] = p
            out.append(x)
    up = torch.arange(V) / V
    out += [up * 0.01, up * 3, up * 90, -up * 20, torch.randn(V, generator=g) * 2.5,
            torch.randn(V, generator=g) + 1e4, (torch.randn(V, generator=g) * 4).round(),
            torch.where(torch.arange(V) % 1024 == 0, 5.0, 0.1234)]
    return torch.stack(out).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1000, 32000, 50001, 150000])
def test_the_logarithm_of_rows_that_round_alike(V, dtype):
    """Scores that leave a best candidate near 0 show it to its last bits."""
    z = rows(V, dtype)
    true = torch.tensor([far(x) for x in z], dtype=torch.float64)
    scores = (-true).float().view(-1, 1).cuda()
    c = scores.double().cpu().flatten() + true
    for a, s in ((z[:, None], scores), (z, scores)):
        got, _, token = fm.beam_select(a, s, 1)
        assert token.flatten().tolist() == first_best(z)
        err = (got.double().cpu().flatten() - c).abs()
        assert (err <= bound(V)).all(), (err.max(), int(err.argmax()))
    # many beams of one element share its blocks another way
    m = 24
    got, parent, _ = fm.beam_select(z[None, :m], scores.view(1, -1)[:, :m].contiguous(), m)
    got, parent = got.double().cpu().flatten(), parent.cpu().flatten()
    own = torch.tensor([c[p] for p in parent.tolist()])
    best = [parent.tolist().index(k) if k in parent else None for k in range(m)]
    for k, i in enumerate(best):
        if i is not None:
            assert abs(float(got[i] - own[i])) <= bound(V)


def nearly(a, b, want, V):
    """Scores (s, t) of beams with rows a and b, whose best candidates are about `want` apart,
    and the gap that they really have."""
    da, db = far(a), far(b)
    s = np.float32(-da)
    t = np.float32(float(s) + da - db - want)
    return float(s), float(t), (float(s) + da) - (float(t) + db)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [700, 32000, 50001])
def test_candidates_of_two_beams_that_are_close(V, dtype):
    """Decided as in 64 bits down to gaps of twice 2^-29, at the border of the selection and in
    its order, whichever beam comes first."""
    z = rows(V, dtype)
    picks = [(2, 9), (1, 41), (5, 14), (0, 7), (25, 44), (38, 40), (11, 3), (43, 46)]
    seen = 0
    for i, j in picks:
        for want in (0.0, 1e-8, 3e-8, 1e-7, 5e-7, 2e-6, -1e-8, -1e-7, -1e-6):
            s, t, gap = nearly(z[i], z[j], want, V)
            if abs(gap) < 2.5 * FINE:
                continue
            seen += abs(gap) < bound(V)
            for pair, sc in (((i, j), (s, t)), ((j, i), (t, s))):
                first = 0 if (gap > 0) == (pair[0] == i) else 1
                a = z[list(pair)][None]
                scores = torch.tensor([sc], dtype=F32, device="cuda")
                assert scores.double().tolist()[0] == list(sc)
                top = first_best(a[0])
                _, parent, token = fm.beam_select(a, scores, 1)
                assert parent.tolist() == [[first]] and token.tolist() == [[top[first]]]
                wide = torch.full((1, 5, V), -math.inf, device="cuda").to(dtype)
                wide[:, 1], wide[:, 4] = a[:, 0], a[:, 1]
                sw = torch.tensor([[0.0, sc[0], -math.inf, 3.0, sc[1]]], device="cuda")
                _, parent, token = fm.beam_select(wide, sw, 1)
                assert parent.tolist() == [[(1, 4)[first]]]
    assert seen > 20


def test_close_candidates_in_the_middle_of_many():
    """Every candidate's place, against 64 bits, of beams whose candidates lie within 1e-6 of
    one another all along."""
    V, n = 20000, 32
    g = torch.Generator().manual_seed(4)
    a = torch.randn(V, generator=g) * 2
    b = a.clone()
    b[torch.randperm(V, generator=g)[:V // 2]] -= 6.0  # another sum under the same peaks
    keep = a.topk(40).indices
    b[keep] = a[keep]
    z = torch.stack([a, b, a + 2.0])[None].cuda()
    da, db = far(z[0, 0]), far(z[0, 1])
    for d in (3e-7, -3e-7, 1e-6, -4e-8):
        s = np.float32(-1.0)
        t = np.float32(float(s) + da - db + d)
        sc = torch.tensor([[float(s), float(t), -1.5]], dtype=F32)
        for m in (1, 2, 7, 31, n):
            want = serve.beam_select(z, sc, m)
            got = fm.beam_select(z, sc.cuda(), m)
            assert got[1].tolist() == want[1].tolist() and got[2].tolist() == want[2].tolist()


def test_close_finished_beams_and_equal_rows():
    V = 9000
    z = torch.randn(V, generator=torch.Generator().manual_seed(2)) * 2
    da = far(z)
    a = z.expand(1, 4, V).contiguous().cuda()
    even = torch.zeros(1, 4, device="cuda")
    _, parent, token = fm.beam_select(a, even, 8)
    top = z.topk(2).indices.tolist()
    assert parent.tolist() == [[0, 1, 2, 3] * 2]
    assert token.tolist() == [[top[0]] * 4 + [top[1]] * 4]
    # a finished beam's score beside a live beam's best candidate
    for d in (2e-8, -2e-8, 3e-7, -3e-7):
        s = np.float32(-da)
        f = np.float32(float(s) + da + d)
        gap = float(f) - (float(s) + da)
        if abs(gap) < 2.5 * FINE:
            continue
        sc = torch.tensor([[float(s), float(f), -math.inf, -math.inf]], dtype=F32, device="cuda")
        fin = torch.tensor([[False, True, False, False]], device="cuda")
        _, parent, token = fm.beam_select(a, sc, 2, finished=fin, pad=5)
        want = [[1, 0], [5, top[0]]] if gap > 0 else [[0, 1], [top[0], 5]]
        assert [parent[0].tolist(), token[0].tolist()] == want
    # finished beams alone, equal ones too
    fin = torch.ones(1, 4, dtype=torch.bool, device="cuda")
    sc = torch.tensor([[-1.0, -0.5, -0.5, -1.0 + 2.0 ** -23]], device="cuda")
    _, parent, token = fm.beam_select(a, sc, 4, finished=fin, pad=5)
    assert parent.tolist() == [[1, 2, 3, 0]] and token.tolist() == [[5] * 4]


def test_close_rows_with_masks_and_in_a_captured_call():
    V = 5000
    g = torch.Generator().manual_seed(8)
    z = torch.randn(6, 3, V, generator=g)
    z[:, 0, 100:] = -math.inf
    z[:, 1, ::2] = torch.finfo(F32).min
    z[:, 2] *= 0.01
    s = torch.zeros(6, 3)
    for b in range(6):
        for k in range(3):
            s[b, k] = -far(z[b, k])  # all best candidates within 1e-6 of 0
    want = [np.argmax([float(s[b, k]) + far(z[b, k]) for k in range(3)]) for b in range(6)]
    gaps = [sorted(float(s[b, k]) + far(z[b, k]) for k in range(3)) for b in range(6)]
    assert all(x[2] - x[1] > 2.5 * FINE for x in gaps)
    z, s = z.cuda(), s.cuda()
    got = fm.beam_select(z, s, 1)
    assert got[1].flatten().tolist() == want
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fm.beam_select(z, s, 1)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, got))


@pytest.mark.parametrize("B,K,V", [(1, 32, 3000), (7, 9, 2500), (60, 2, 4001), (100, 5, 900),
                                   (200, 32, 1100)])
def test_close_candidates_however_an_element_is_cut(B, K, V):
    """All beams' best candidates within some 1e-6, on clusters of 8 blocks down to one."""
    g = torch.Generator().manual_seed(B)
    z = torch.randn(B, K, V + 3, generator=g).to(BF16)[:, :, 3:]
    zd = z.double()
    lse = torch.logsumexp(zd, 2)
    top = zd.amax(2)
    s = (lse - top + 1e-6 * torch.randn(B, K, generator=g).double()).float()
    best, order = torch.sort(s.double() + (top - lse), 1, descending=True)
    n = min(K, 4)
    gap = best[:, :n] - torch.cat([best[:, 1:], torch.full((B, 1), -1.0)], 1)[:, :n]
    # second candidates of a beam lie in between where a row has its maximum twice
    alone = ((zd == top[..., None]).sum(2) == 1).all(1) & (gap > 2.5 * FINE).all(1)
    assert alone.double().mean() > 0.5 or K > 8
    wide = torch.zeros(B, K, V + 3, dtype=BF16, device="cuda")
    wide[:, :, 3:] = z.cuda()
    score, parent, token = fm.beam_select(wide[:, :, 3:], s.cuda(), n)
    want = torch.gather(zd.argmax(2), 1, order)[:, :n]
    assert torch.equal(parent.cpu()[alone], order[:, :n][alone])
    assert torch.equal(token.cpu()[alone], want[alone])
    err = (score.cpu().double() - best[:, :n]).abs()[alone]
    assert alone.any() and (err <= bound(V)).all()
