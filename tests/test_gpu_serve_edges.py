"""Generation with states at its edges: offsets behind 2^31, many heads and tiles, calls on
several streams and threads at once, graphs that are replayed side by side, and work that
is queued behind the writers of its operands."""
import math
import threading

import numpy as np
import pytest
import torch

import flash_mixed_chunk_gb300 as fm
from oracle import serve

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rand(*s, dtype=BF16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + len(s) + s[-1])
    return torch.randn(*s, generator=g, device="cuda").to(dtype)


def settled():
    torch.cuda.synchronize()
    assert fm.flash_mca_device_status()[0] == fm.FMCA_OK


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F32, 20)])
def test_operands_and_outputs_behind_2_to_31(dtype, d):
    """A batch whose second sequence lies 2^31 elements behind the first, and outputs of more
    than 2^31 elements: the same values as apart."""
    T, H, far = 300, 2, 2 ** 31 + 64
    buf = torch.empty(far + T * H * d, dtype=dtype, device="cuda")
    x = rand(2, T, H, d, dtype=dtype)
    view = torch.as_strided(buf, (2, T, H, d), (far, H * d, d, 1))
    view.copy_(x)
    ld = torch.tensor([-0.02, -0.3]).cuda()
    want, ws = fm.decay_attention(x, x, x, ld)
    got, gs = fm.decay_attention(view, view, view, ld)
    settled()
    assert torch.equal(want, got) and torch.equal(ws, gs)
    # one step from there, q, k and v as far apart
    s1, s2 = ws.clone(), ws.clone()
    a = fm.decay_step(x[:, 5], x[:, 6], x[:, 7], ld, s1)
    b = fm.decay_step(view[:, 5], view[:, 6], view[:, 7], ld, s2)
    settled()
    assert torch.equal(a, b) and torch.equal(s1, s2)


def test_states_behind_2_to_31():
    """A state of more than 2^31 elements: its last sequences as they are apart."""
    B, H, dk, dv = 2 ** 31 // (16 * 128 * 128) + 3, 16, 128, 128
    state = torch.zeros(B, H, dk, dv, device="cuda")
    q, k, v = rand(B, H, dk), rand(B, H, dk, seed=1), rand(B, H, dv, seed=2)
    ld = -torch.rand(H, device="cuda")
    state[-2:] = rand(2, H, dk, dv, dtype=F32)
    small = state[-2:].clone()
    o = fm.decay_step(q, k, v, ld, state)
    p = fm.decay_step(q[-2:], k[-2:], v[-2:], ld, small)
    settled()
    assert torch.equal(state[-2:], small)  # each element is of two products, in one order
    # o sums dk products, in an order that depends on how many states there are: either sum
    # is within (dk + 2) 2^-24 of the products' sizes, and either rounds to bf16 (2^-8)
    size = torch.einsum("bhk,bhkv->bhv", q[-2:].double().abs(), small.double().abs())
    a, b = o[-2:].double(), p.double()
    assert ((a - b).abs() <= 2 * (dk + 2) * 2.0 ** -24 * size
            + 2.0 ** -8 * (a.abs() + b.abs())).all()
    o, out = fm.decay_attention(q[:, None], k[:, None], v[:, None], ld, state=state)
    p, s = fm.decay_attention(q[-2:, None], k[-2:, None], v[-2:, None], ld, state=small)
    settled()
    assert torch.equal(o[-2:], p) and torch.equal(out[-2:], s)


def test_logits_and_rows_behind_2_to_31():
    K, V = 4, 32768
    B = 2 ** 31 // (K * V) + 2
    z = torch.empty(B, K, V, dtype=BF16, device="cuda")
    z.fill_(-1.0)
    z[-2:] = rand(2, K, V)
    scores = -torch.arange(B * K, device="cuda").view(B, K).remainder(7).float()
    got = fm.beam_select(z, scores, 8)
    want = fm.beam_select(z[-2:], scores[-2:], 8)
    settled()
    assert all(torch.equal(a[-2:], b) for a, b in zip(got, want))
    del z
    rows = torch.zeros(8, 2 ** 29, device="cuda")  # 2 GiB apart
    rows[:, :100] = rand(8, 100, dtype=F32)
    parent = torch.tensor([[3, 3, 0, 1], [2, 1, 0, 3]], device="cuda")
    want = torch.as_tensor(serve.reorder(rows[:, :100].cpu(), parent.tolist()))
    fm.beam_reorder([rows[:, :100]], parent)
    settled()
    assert torch.equal(rows[:, :100].cpu(), want) and not rows[:, 100:200].any()


@pytest.mark.parametrize("B,T,H,dk,dv,dtype", [
    (3, 130, 120, 16, 24, BF16), (40, 33, 8, 64, 64, BF16), (1, 140, 2, 24, 2000, BF16),
    (1, 70, 2, 7, 1030, F32), (300, 2, 2, 8, 8, BF16), (1, 20000, 1, 16, 16, BF16),
    (1, 9000, 1, 9, 10, F32)])
def test_many_heads_tiles_and_segments(B, T, H, dk, dv, dtype):
    q, k, v = rand(B, T, H, dk, dtype=dtype), rand(B, T, 1, dk, dtype=dtype, seed=1), \
        rand(B, T, H, dv, dtype=dtype, seed=2)
    ld = -math.log(2) / torch.linspace(3, 900, H).cuda()
    o, s = fm.decay_attention(q, k, v, ld, scale=0.25)
    settled()
    pick = [0, B - 1] if B > 1 else [0]
    heads = sorted({0, H // 2, H - 1})
    ro, rs, sz = serve.decay_attention(q[pick][:, :, heads], k[pick], v[pick][:, :, heads],
                                       ld[heads], None, 0.25)
    tol = (2 * dk + T + 64) * 2.0 ** -23 * sz["whole"]
    if dtype == BF16:
        tol += 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -16) * (sz["near"] + sz["far"])
    got = o[pick][:, :, heads].float().cpu().numpy()
    assert (np.abs(got - ro) <= tol).all()
    got = s[pick][:, heads].cpu().numpy()
    assert (np.abs(got - rs) <= (3 * T + 64) * 2.0 ** -23 * sz["state"]).all()


def calls(seed):
    """One of each call, on operands of its own: (call, results that it has to give)."""
    H, d = 3, 64
    q, k, v = (rand(2, 700, H, d, seed=seed + i) for i in range(3))
    ld = torch.tensor([-0.01, -0.1, -1.0]).cuda()
    s0 = rand(2, H, d, d, dtype=F32, seed=seed)
    z, sc = rand(2, 4, 5003, seed=seed, dtype=F32), -torch.rand(2, 4, device="cuda")
    rows = rand(8, 3000, dtype=F32, seed=seed)
    parent = torch.tensor([[1, 0, 3, 3], [0, 0, 2, 1]], device="cuda")
    back = torch.tensor([[0, 1, 2, 3], [0, 1, 2, 3]], device="cuda")

    def call():
        o, s = fm.decay_attention(q, k, v, ld, state=s0)
        y = fm.decay_step(q[:, 0], k[:, 1], v[:, 2], ld, s)
        picked = fm.beam_select(z, sc, 6)
        t = rows.clone()
        fm.beam_reorder([t], parent)
        fm.beam_reorder([t], back)
        return [o, s, y, *picked, t]

    return call


def test_streams_and_threads_at_once():
    made = [calls(10 * i) for i in range(4)]
    want = [c() for c in made]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    got[i] = made[i]()
            stream.synchronize()
        except Exception as exc:  # seen by the test's thread
            errors.append(exc)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    settled()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_graphs_side_by_side():
    """Two captured runs replayed on two streams, at once and alternately: each has the
    workspace of its own capture."""
    made = [calls(100), calls(200)]
    want = [c() for c in made]
    torch.cuda.synchronize()
    graphs, got = [], []
    for c in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(c())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    settled()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_behind_the_writers_of_the_operands():
    """Operands that a long-running kernel, a copy or a memset ahead on the stream writes
    last, and outputs that the next one overwrites."""
    H, d, T = 2, 64, 1500
    src = [rand(1, T, H, d, seed=i) for i in range(3)]
    ld = torch.tensor([-0.02, -0.2]).cuda()
    want, ws = fm.decay_attention(*src, ld)
    z = rand(2, 4, 9001, dtype=F32)
    sc = -torch.rand(2, 4, device="cuda")
    ws3 = fm.beam_select(z, sc)
    torch.cuda.synchronize()
    heavy = torch.randn(4096, 4096, device="cuda")
    for _ in range(5):
        q, k, v = (torch.full_like(x, 9.0) for x in src)
        z2, sc2 = torch.zeros_like(z), torch.zeros_like(sc)
        torch.mm(heavy, heavy)
        for a, b in zip((q, k, v, z2, sc2), (*src, z, sc)):
            a.copy_(b)
        o, s = fm.decay_attention(q, k, v, ld)
        got = fm.beam_select(z2, sc2)
        kept = o.clone(), s.clone(), [g.clone() for g in got]
        for t in (q, k, v, z2, sc2, o, s, *got):
            t.zero_()
        settled()
        assert torch.equal(kept[0], want) and torch.equal(kept[1], ws)
        assert all(torch.equal(a, b) for a, b in zip(kept[2], ws3))


def test_lengths_change_under_a_captured_call():
    q, k, v = (rand(3, 500, 2, 64, seed=i) for i in range(3))
    ld = torch.tensor([-0.02, -0.2]).cuda()
    lengths = torch.tensor([500, 1, 0], dtype=torch.int32, device="cuda")
    fm.decay_attention(q, k, v, ld, lengths=lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = fm.decay_attention(q, k, v, ld, lengths=lengths)
    for new in ([500, 1, 0], [3, 499, 128], [0, 0, 0], [600, -1, 129]):
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        p, t = fm.decay_attention(q, k, v, ld, lengths=lengths)
        settled()
        assert torch.equal(o, p) and torch.equal(s, t)


@pytest.mark.parametrize("dtype,T,dk,dv", [(BF16, 200, 64, 64), (BF16, 300, 128, 200),
                                           (BF16, 2000, 16, 72), (F32, 150, 20, 70)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite_reach_no_earlier_row(dtype, T, dk, dv, bad):
    """An infinity or NaN in a token's q, k or v reaches its own and later rows alone, one
    in v its own column alone: all others are as without it, bit for bit."""
    q, k, v = rand(2, T, 2, dk, dtype=dtype), rand(2, T, 2, dk, dtype=dtype, seed=1), \
        rand(2, T, 2, dv, dtype=dtype, seed=2)
    ld = torch.tensor([-0.02, -0.5]).cuda()
    want, ws = fm.decay_attention(q, k, v, ld)
    for t, c in ((T - 1, 0), (T // 2 + 3, dv - 1), (5, 9), (127, 33), (128, 63), (1, 15)):
        x = v.clone()
        x[0, t, 1, c] = bad
        o, s = fm.decay_attention(q, k, x, ld)
        settled()
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[0, t:, 1, c] = True
        assert torch.equal(o[~hit], want[~hit])
        assert not torch.isfinite(o[0, t, 1, c])
        hit = torch.zeros_like(s, dtype=torch.bool)
        hit[0, 1, :, c] = True
        assert torch.equal(s[~hit], ws[~hit]) and not torch.isfinite(s[hit]).any()
    # two columns and three rows of one, at once
    x = v.clone()
    x[0, 40, 0, 2], x[0, 60, 0, 2], x[1, 90, 1, 3], x[0, 50, 0, 3] = bad, 1.0, bad, bad
    o, _ = fm.decay_attention(q, k, x, ld)
    settled()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, 40:, 0, 2] = hit[1, 90:, 1, 3] = hit[0, 50:, 0, 3] = hit[0, 60:, 0, 2] = True
    assert torch.equal(o[~hit], want[~hit])
    for t in (0, 77, 128, T - 1):
        x = k.clone()
        x[1, t, 0, dk - 1] = bad
        o, s = fm.decay_attention(q, x, v, ld)
        settled()
        assert torch.equal(o[0], want[0]) and torch.equal(s[0], ws[0])
        assert torch.equal(o[1, :, 1], want[1, :, 1])
        assert torch.equal(o[1, :t, 0], want[1, :t, 0])
        assert not torch.isfinite(o[1, t, 0]).any()
        x = q.clone()
        x[1, t, 0, 0] = bad
        o, s = fm.decay_attention(x, k, v, ld)
        settled()
        rest = torch.ones_like(o, dtype=torch.bool)
        rest[1, t, 0] = False
        assert torch.equal(o[rest], want[rest]) and torch.equal(s, ws)


def test_the_longest_row_of_logits():
    V = 2 ** 31 - 1
    z = torch.zeros(1, 1, V, dtype=BF16, device="cuda")
    at = [V - 1, 2 ** 30 + 5, 3]
    z[0, 0, at] = torch.tensor([9.0, 8.0, 8.0], dtype=BF16, device="cuda")
    score, parent, token = fm.beam_select(z, torch.zeros(1, 1, device="cuda"), 4)
    settled()
    assert token.tolist() == [[V - 1, 3, 2 ** 30 + 5, 0]] and not parent.any()
    lse = math.log(V - 3 + math.exp(9.0) + 2 * math.exp(8.0))
    # a sum of V equal terms of 1 by lanes, warps and blocks: 32 lanes' and 32 places' sums
    # are exact up to 2^24, what is added to them late loses at most half a step of 2^31 / 2^24
    # each (2^-24 of it), over V / 1024 / 8 / 8 turns of a warp of 64
    turns = V / 1024 / 64
    got = torch.tensor([9.0, 8.0, 8.0, 0.0], dtype=torch.float64) - lse
    assert ((score[0].cpu().double() - got).abs() <= (turns + 70) * 2.0 ** -24 + 2.0 ** -19).all()


def test_rows_that_overlap_and_other_orders():
    """Tokens closer than their rows are long, heads inside one another, tokens innermost but
    for the row, batches last: as contiguous copies of them, bit for bit."""
    B, T, H, d = 2, 300, 3, 64
    flat = rand(B * T * H * d)
    views = [
        torch.as_strided(flat, (B, T, H, d), (T * 8, 8, 16, 1)),
        torch.as_strided(flat, (B, T, H, d), (8, 24, 64, 1)),
        flat.view(B, H, T, d).transpose(1, 2),
        flat.view(H, T, B, d).permute(2, 1, 0, 3),
        flat.view(T, H, B, d).permute(2, 0, 1, 3),
    ]
    ld = torch.tensor([-0.01, -0.1, -0.7]).cuda()
    for x in views:
        for y in (views[2], x):
            want = fm.decay_attention(x.contiguous(), x.contiguous(), y.contiguous(), ld)
            got = fm.decay_attention(x, x, y, ld)
            settled()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
            s1, s2 = want[1].clone(), want[1].clone()
            a = fm.decay_step(x[:, 3], x[:, 4], y[:, 5], ld, s1)
            b = fm.decay_step(x[:, 3].contiguous(), x[:, 4].contiguous(), y[:, 5].contiguous(), ld,
                              s2)
            assert torch.equal(a, b) and torch.equal(s1, s2)
