"""Linear attention with log decays above 0: a state that grows past the range of 32 bits."""
import math

import pytest
import torch

import flash_mixed_chunk_gb300 as fm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(B, T, H, dk, dv, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    q, k, v = (torch.randn(B, T, H, d, generator=g).to(dtype).cuda() for d in (dk, dk, dv))
    return q, k, v, torch.randn(B, H, dk, dv, generator=g).cuda()


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
