"""Calls of generation with states that are easily got wrong: strided logits of two
dimensions, too many candidates, pieces whose rows lie inside one another,
tensors that autograd has saved."""
import pytest
import torch

import flash_mixed_chunk_gb300 as fm

pytestmark = pytest.mark.gpu


def test_logits_of_two_dimensions_have_a_row_for_each_beam():
    """A column of a matrix is [1, 4] with scores [1, 4], but not the logits of 4 beams."""
    w = torch.randn(4, 4, device="cuda")
    scores = torch.zeros(1, 4, device="cuda")
    out = (torch.empty(1, 4, device="cuda"),
           *(torch.empty(1, 4, dtype=torch.int64, device="cuda") for _ in range(2)))
    for bad in (w[:, 3][None], w[:, 0][None], w[:1], torch.randn(2, 4, device="cuda")[1:]):
        with pytest.raises(ValueError):
            fm.beam_select(bad, scores)
        with pytest.raises(ValueError):
            fm.flash_mca_beam_select(bad, scores, None, *out)
    one = torch.randn(3, 7, device="cuda")[:, :5]  # [B, V] for single beams stays a call
    got = fm.beam_select(one, torch.zeros(3, 1, device="cuda"))
    assert got[2].flatten().tolist() == one.argmax(1).tolist()
    got = fm.beam_select(torch.randn(1, 1, device="cuda"), scores[:, :1])
    assert got[2].tolist() == [[0]]


def test_too_many_candidates_are_refused_before_memory_is_taken():
    logits, scores = torch.zeros(8, 4, 50, device="cuda"), torch.zeros(8, 4, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for n in (33, 10 ** 6, 2 ** 31 - 1):
        with pytest.raises(fm.FmcaError):
            fm.beam_select(logits, scores, n)
    many = torch.zeros(1, 40, 5, device="cuda")  # 40 beams, and so 40 candidates by default
    before += many.numel() * 4 + 2048
    with pytest.raises(fm.FmcaError):
        fm.beam_select(many, many[:, :, 0].contiguous())
    assert torch.cuda.max_memory_allocated() <= before


@pytest.mark.parametrize("call", ["beam_reorder", "flash_mca_beam_reorder"])
def test_rows_inside_one_another(call):
    """Column ranges of one buffer are pieces that share no byte; parent may lie between
    rows, too."""
    g = torch.Generator().manual_seed(1)
    parent = torch.tensor([[1, 1, 3, 0], [2, 2, 0, 3]], device="cuda")
    rows = (parent + 4 * torch.arange(2, device="cuda")[:, None]).flatten()
    reorder = getattr(fm, call)
    buf = torch.randn(8, 200, generator=g).cuda()
    want = buf[rows]
    reorder([buf[:, :100], buf[:, 100:]], parent)
    assert torch.equal(buf, want)
    want = buf.clone()
    want[:, 150:190], want[:, 3:77] = buf[rows, 150:190], buf[rows, 3:77]
    reorder([buf[:, 150:190], buf[:, 3:50], buf[:, 50:77]], parent)
    assert torch.equal(buf, want)
    wrap = torch.randn(8 * 20 + 30, generator=g).cuda()  # the second piece a row further on
    a, b = torch.as_strided(wrap, (8, 12), (20, 1), 0), torch.as_strided(wrap, (8, 8), (20, 1), 32)
    wa, wb = a[rows], b[rows]
    reorder([b, a], parent)
    assert torch.equal(a, wa) and torch.equal(b, wb)
    # parent between the rows of a piece, as 16 bytes of one beam in a buffer of 64-bit numbers
    own = torch.zeros(4, 12, dtype=torch.int64, device="cuda")
    own[:, 8:] = torch.arange(16, device="cuda").view(4, 4)
    near = torch.as_strided(own, (1, 4), (48, 1), 0)
    near.copy_(torch.tensor([[3, 2, 2, 0]]))
    part = own[:, 4:]
    wp = part[near[0]]
    reorder([part], near)
    assert torch.equal(part, wp) and near.tolist() == [[3, 2, 2, 0]]
    for bad in ([own], [own[:, 3:5]]):
        with pytest.raises(fm.FmcaError):
            reorder(bad, near)
    for bad in ([buf[:, :100], buf[:, 99:]], [buf[:, 50:60], buf[:, :51]], [buf, buf[:, 7:8]],
                [a, torch.as_strided(wrap, (8, 9), (20, 1), 32)],
                [buf[:, :100], torch.as_strided(buf, (8, 10), (150, 1), 100)]):
        with pytest.raises(fm.FmcaError):
            reorder(bad, parent)


def test_writes_are_seen_by_autograd():
    """A tensor that a backward pass has saved and a call overwrites is an error there."""
    B, K, H, d = 1, 4, 2, 16
    q = torch.randn(B * K, H, d, device="cuda")
    ld = torch.tensor([-0.1, -0.2], device="cuda")
    parent = torch.tensor([[1, 0, 2, 2]], device="cuda")
    x = torch.randn(B, K, 50, device="cuda")
    scores = torch.zeros(B, K, device="cuda")
    idx = lambda: torch.zeros(B, K, dtype=torch.int64, device="cuda")  # noqa: E731
    core = torch.zeros(fm.flash_mca_decode_state_bytes(B * K, 8, 8, 16, fm.FMCA_F32),
                       dtype=torch.uint8, device="cuda")
    state = torch.randn(B * K, H, d, d, device="cuda")
    o = torch.empty(B * K, H, d, device="cuda")
    row = torch.randn(B * K, 30, device="cuda")
    half = torch.randn(B * K, 30, device="cuda")
    out = torch.empty(B, K, device="cuda"), idx(), idx()
    prompt = [t[None] for t in (q, q, q)]
    po, ps = torch.empty(1, B * K, H, d, device="cuda"), torch.empty(1, H, d, d, device="cuda")
    for written, call in [
            ([state], lambda: fm.decay_step(q, q, q, ld, state)),
            ([state, o], lambda: fm.flash_mca_decay_step(q, q, q, ld, state, o)),
            ([po, ps], lambda: fm.flash_mca_decay_attention(*prompt, ld, None, None, po, ps, None)),
            ([po], lambda: fm.flash_mca_decay_attention(*prompt, ld, None, ps, po, None, None)),
            ([row, half], lambda: fm.beam_reorder([row, half[:, :7]], parent)),
            ([row, half], lambda: fm.flash_mca_beam_reorder([row, half[:, :7]], parent)),
            (list(out), lambda: fm.flash_mca_beam_select(x, scores, None, *out)),
            ([core], lambda: fm.flash_mca_decode_reorder(core, parent, 8, 8, 16, 3, fm.FMCA_F32))]:
        before = [t._version for t in written]
        call()
        assert all(t._version > v for t, v in zip(written, before))
    read = [q, ld, parent, x, scores]
    assert not any(t._version for t in read)
    w = torch.randn(B * K, H, d, d, device="cuda", requires_grad=True)
    y = (w * state).sum()
    fm.decay_step(q, q, q, ld, state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    v = state._version
    with pytest.raises(ValueError):
        fm.decay_step(q, q, q, ld, state[:1])
    assert state._version == v  # a call that is refused writes nothing
    with torch.inference_mode():  # tensors without a version
        s = torch.zeros_like(state)
        fm.decay_step(q, q, q, ld, s)
        fm.beam_reorder([s], parent)
        fm.flash_mca_decay_step(q, q, q, ld, s, o)
    torch.cuda.synchronize()
