"""Calls of generation with states that are easily got wrong: strided logits of two
dimensions, too many candidates."""
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
