"""Shapes and pieces of generation with states that the wrappers tell apart (CPU)."""
import pytest
import torch

import flash_mixed_chunk_gb300 as fm


def test_rows_of_logits():
    """A [1, 4] view whose elements lie apart is no [4, 4]: its rows would end behind it."""
    w = torch.zeros(4, 4)
    for bad, B, K in ((w[:, 3][None], 1, 4), (w[:1], 1, 4), (torch.zeros(2, 3, 5), 3, 2),
                      (torch.zeros(6, 5), 2, 2), (torch.zeros(4), 1, 4), (w.t(), 4, 1),
                      (torch.zeros(2, 2, 1, 5), 2, 2)):
        with pytest.raises(ValueError):
            fm._logit_row(bad, B, K)
    for good, B, K, row in ((w, 1, 4, 4), (w, 2, 2, 4), (torch.zeros(3, 9)[:, :5], 3, 1, 9),
                            (torch.zeros(2, 3, 9)[..., :5], 2, 3, 9), (w[:1, :3], 1, 1, 3),
                            (torch.zeros(4, 7)[:, 2:3], 2, 2, 7), (torch.zeros(1, 1), 1, 1, 1),
                            (torch.zeros(2, 5, 3)[:, 0], 1, 2, 15)):
        assert fm._logit_row(good, B, K) == row


def test_pieces_that_share_a_byte_are_refused():
    """Rows inside one another: [first, first + bytes) of every row, also over a row's end."""
    P = 1 << 20  # a made-up device address, never read

    def status(*pieces, parent=1 << 40, B=2, K=4):
        p = (fm.FmcaBeamPiece * len(pieces))(*[fm.FmcaBeamPiece(*x) for x in pieces])
        return fm.lib.flash_mca_beam_reorder(p, len(pieces), parent, B, K, None)

    for pieces in (((P, 800, 400), (P + 399, 800, 401)), ((P + 399, 800, 401), (P, 800, 400)),
                   ((P, 80, 48), (P + 128, 80, 33)), ((P + 128, 80, 33), (P, 80, 48)),
                   ((P, 80, 48), (P + 48, 81, 20)), ((P, 80, 48), (P + 600, 80, 40)),
                   ((P, 80, 80), (P + 79, 80, 1)), ((P, 80, 1), (P - 160, 80, 1))):
        assert status(*pieces) == fm.FMCA_ERR_INVALID_ARG, pieces
    for parent in (P + 40, P - 8, P + 8 * 96 - 72, P + 24 + 96):
        assert status((P, 96, 32), parent=parent) == fm.FMCA_ERR_INVALID_ARG
