"""Linear attention with a decay for each head on the GPU against the fp64 oracle.

Bounds, an element at a time, with the oracle's sums of absolute values (oracle.serve):
bf16 outputs round once, and the tensor-core kernel rounds a chunk's weights and the
state as an operand, each by half a step (2^-8 of the value): 2^-8 (|o| + near + far),
where a second rounding of a rounded value adds 2^-16 of it.  fp32 sums of N terms are
off by at most N 2^-23 of the sum of absolute values (2^-23: a tensor core's sum may cut
instead of round); a term passes through the dk products of q k, the at most T of a
chunk or of the state, the dk of q S and two powers, each within 2^-21.  Where a state is
multiplied by a power once a chunk, it is by two floats (2^-46).
"""
import math

import numpy as np
import pytest
import torch

import flash_mixed_chunk_gb300 as fm
from oracle import serve

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(B, T, H, Hq, Hk, Hv, dk, dv, dtype, seed=0, packed=False, fast=4.0, slow=400.0):
    g = torch.Generator().manual_seed(1000 * seed + T)
    sizes = [(Hq, dk), (Hk, dk), (Hv, dv)]
    if packed:
        rows = torch.randn(B, T, sum(h * d for h, d in sizes), generator=g).to(dtype).cuda()
        q, k, v = (p.unflatten(-1, s)
                   for p, s in zip(rows.split([h * d for h, d in sizes], -1), sizes))
    else:
        q, k, v = (torch.randn(B, T, *s, generator=g).to(dtype).cuda() for s in sizes)
    half = fast * (slow / fast) ** torch.rand(H, generator=g)
    ld = (-math.log(2) / half).cuda()
    state = torch.randn(B, H, dk, dv, generator=g).cuda() * 3
    return q, k, v, ld, state


def check_o(o, ref, size, dk, T, dtype, prompt=True):
    o = o.float().cpu().numpy()
    assert not np.isnan(o).any()
    tol = (2 * dk + T + 64) * 2.0 ** -23 * size["whole"]
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
        if prompt:
            tol = tol + (2.0 ** -8 + 2.0 ** -16) * (size["near"] + size["far"])
    err = np.abs(o - ref) - tol
    assert (err <= 0).all(), (err.max(), np.unravel_index(err.argmax(), err.shape))


def check_state(s, ref, size, T):
    tol = (3 * T + 64) * 2.0 ** -23 * size["state"]
    assert (np.abs(s.cpu().numpy() - ref) <= tol).all()


def settled():
    torch.cuda.synchronize()
    assert fm.flash_mca_device_status()[0] == fm.FMCA_OK


# B, T, H, Hq, Hk, Hv, dk, dv
SIZES = [
    (1, 1, 1, 1, 1, 1, 8, 8), (2, 3, 2, 2, 2, 2, 64, 64), (1, 37, 4, 4, 4, 4, 64, 64),
    (2, 127, 2, 1, 2, 2, 128, 128), (1, 128, 3, 3, 1, 3, 128, 64), (1, 129, 2, 2, 2, 1, 64, 128),
    (2, 300, 6, 2, 3, 6, 40, 72), (1, 1000, 2, 1, 1, 2, 128, 128), (1, 2100, 1, 1, 1, 1, 96, 120),
    (3, 257, 2, 2, 2, 2, 16, 200), (1, 515, 2, 2, 1, 1, 24, 136),
    (2, 70, 3, 3, 3, 3, 37, 75), (1, 600, 2, 2, 2, 2, 5, 3), (1, 90, 2, 1, 1, 2, 200, 264),
    (1, 33, 1, 1, 1, 1, 256, 31), (2, 65, 2, 2, 2, 2, 1, 1), (1, 700, 1, 1, 1, 1, 130, 65),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", SIZES)
def test_prompts(size, dtype):
    q, k, v, ld, state = make(*size, dtype)
    T, dk = size[1], size[6]
    for s0 in (None, state):
        o, s = fm.decay_attention(q, k, v, ld, state=s0, scale=0.3)
        settled()
        ro, rs, sz = serve.decay_attention(q, k, v, ld, s0, 0.3)
        assert o.dtype == dtype and s.dtype == F32
        check_o(o, ro, sz, dk, T, dtype)
        check_state(s, rs, sz, T)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (40, 75)])
def test_lengths_and_what_lies_behind(dk, dv, dtype):
    B, T, H = 7, 390, 3
    q, k, v, ld, state = make(B, T, H, 3, 1, 3, dk, dv, dtype, packed=dv != 75)
    lengths = torch.tensor([390, 0, 1, 128, 129, 255, 1000], dtype=torch.int32).cuda()
    for b, n in enumerate([390, 0, 1, 128, 129, 255, 390]):
        for t in (q, k, v):
            t[b, n:] = float("nan")
            if n + 1 < T:
                t[b, n + 1:] = float("inf")
    o, s = fm.decay_attention(q, k, v, ld, state=state, lengths=lengths)
    settled()
    ro, rs, sz = serve.decay_attention(q, k, v, ld, state, 1.0, lengths)
    check_o(o, ro, sz, dk, T, dtype)
    check_state(s, rs, sz, T)
    assert torch.equal(s[1], state[1]) and not o[1].any()
    gone, s = fm.decay_attention(q, k, v, ld, lengths=torch.full_like(lengths, -5))
    assert not gone.any() and not s.any()


def test_strides_of_every_kind():
    B, T, H, d = 2, 200, 4, 64
    g = torch.Generator().manual_seed(5)
    base = torch.randn(T, B, H, d, generator=g).to(BF16).cuda()
    ld = torch.tensor([-0.01, -0.1, -0.5, -1.0]).cuda()
    forms = {
        "tokens first": base.transpose(0, 1),
        "heads first": torch.randn(B, H, T, d, generator=g).to(BF16).cuda().transpose(1, 2),
        "one head for all": base[:, :, :1].transpose(0, 1).expand(B, T, H, d),
        "one sequence for all": base.transpose(0, 1)[:1].expand(B, T, H, d),
        "one token for all": base.transpose(0, 1)[:, :1].expand(B, T, H, d),
        "odd offset": torch.randn(B * T * H * d + 3, generator=g).to(BF16).cuda()[3:].view(
            B, T, H, d),
        "odd rows": torch.randn(B, T, H, d + 3, generator=g).to(BF16).cuda()[..., :d],
        "every other token": torch.randn(B, 2 * T, H, d, generator=g).to(BF16).cuda()[:, ::2],
    }
    for name, x in forms.items():
        for q, k, v in ((x, forms["heads first"], base.transpose(0, 1)),
                        (forms["heads first"], x, x), (x, x, x)):
            o, s = fm.decay_attention(q, k, v, ld)
            settled()
            ro, rs, sz = serve.decay_attention(q, k, v, ld)
            check_o(o, ro, sz, d, T, BF16)
            check_state(s, rs, sz, T)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decays_from_none_to_all(dtype):
    q, k, v, _, state = make(1, 500, 6, 6, 6, 6, 64, 64, dtype)
    # no decay; slow; as strong as one chunk's powers underflow; none of the past kept
    ld = torch.tensor([0.0, -1e-4, -0.7, -20.0, -1e4, -math.inf]).cuda()
    o, s = fm.decay_attention(q, k, v, ld, state=state)
    settled()
    ro, rs, sz = serve.decay_attention(q, k, v, ld, state)
    check_o(o, ro, sz, 64, 500, dtype)
    check_state(s, rs, sz, 500)
    o, _ = fm.decay_attention(q, k, v, torch.full_like(ld, math.nan))
    assert o.isnan().all()


def test_a_nan_stays_with_its_head_and_its_future():
    q, k, v, ld, _ = make(2, 300, 2, 2, 2, 2, 64, 64, BF16)
    clean, sc = fm.decay_attention(q, k, v, ld)
    k[1, 150, 0, 3] = math.nan
    o, s = fm.decay_attention(q, k, v, ld)
    assert torch.equal(o[0], clean[0]) and torch.equal(o[1, :, 1], clean[1, :, 1])
    assert torch.equal(o[1, :150, 0], clean[1, :150, 0])
    assert o[1, 150:, 0].isnan().all() and s[1, 0].isnan().any()
    assert torch.equal(s[0], sc[0]) and torch.equal(s[1, 1], sc[1, 1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cut", [1, 100, 128, 300])
def test_pieces_of_a_prompt(cut, dtype):
    q, k, v, ld, state = make(2, 400, 3, 3, 3, 3, 64, 80, dtype)
    ro, rs, sz = serve.decay_attention(q, k, v, ld, state)
    o1, s1 = fm.decay_attention(q[:, :cut], k[:, :cut], v[:, :cut], ld, state=state)
    o2, s2 = fm.decay_attention(q[:, cut:], k[:, cut:], v[:, cut:], ld, state=s1)
    # the second piece's chunks start elsewhere: a bound over both terms at once
    sz = {**sz, "near": sz["whole"], "far": 0 * sz["whole"]}
    check_o(torch.cat([o1, o2], 1), ro, sz, 64, 400, dtype)
    check_state(s2, rs, sz, 400)


@pytest.mark.parametrize("B,T,H", [(1, 5000, 1), (2, 3000, 5)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_segments_in_place_and_workspace(B, T, H, dtype):
    """Few heads and many tokens: the sequence is cut into segments; the state in place."""
    q, k, v, ld, state = make(B, T, H, H, H, H, 64, 64, dtype, slow=4000.0)
    need = fm.flash_mca_decay_workspace_bytes(q, k, v, ld)
    assert need > 0
    lengths = torch.full((B,), T - 700, dtype=torch.int32).cuda()
    want, s = fm.decay_attention(q, k, v, ld, state=state, lengths=lengths)
    ro, rs, sz = serve.decay_attention(q, k, v, ld, state, 1.0, lengths)
    check_o(want, ro, sz, 64, T, dtype)
    check_state(s, rs, sz, T)
    o = torch.full_like(want, 7.0)
    guard = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    place = state.clone()
    fm.flash_mca_decay_attention(q, k, v, ld, lengths, place, o, place, guard[256:-256])
    settled()
    assert torch.equal(o, want) and torch.equal(place, s)
    assert (guard[:256] == 255).all() and (guard[-256:] == 255).all()
    fm.flash_mca_decay_attention(q, k, v, ld, lengths, state, o, None, guard[256:-256])
    settled()
    assert torch.equal(o, want)


def test_same_bits_again_and_captured():
    q, k, v, ld, state = make(2, 1500, 4, 4, 4, 4, 128, 128, BF16)
    o, s = fm.decay_attention(q, k, v, ld, state=state)
    for _ in range(3):
        o2, s2 = fm.decay_attention(q, k, v, ld, state=state)
        assert torch.equal(o, o2) and torch.equal(s, s2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        og, sg = fm.decay_attention(q, k, v, ld, state=state)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, og) and torch.equal(s, sg)
    q.mul_(2.0)
    graph.replay()
    o2, _ = fm.decay_attention(q, k, v, ld, state=state)
    torch.cuda.synchronize()
    assert torch.equal(og, o2)
    settled()


STEPS = [(1, 1, 1, 1, 1, 8, 8), (3, 4, 2, 1, 4, 64, 64), (2, 12, 12, 12, 12, 128, 128),
         (40, 12, 1, 1, 12, 128, 128), (5, 6, 2, 3, 1, 37, 75), (2, 3, 3, 3, 3, 256, 300),
         (7, 2, 2, 1, 2, 1, 1), (1, 1, 1, 1, 1, 200, 6), (200, 2, 2, 2, 2, 100, 132)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", STEPS)
def test_steps(size, dtype):
    B, H, Hq, Hk, Hv, dk, dv = size
    q, k, v, ld, state = make(B, 3, H, Hq, Hk, Hv, dk, dv, dtype)
    ro, rs, sz = serve.decay_attention(q, k, v, ld, state, 0.5)
    o = [fm.decay_step(q[:, t], k[:, t], v[:, t], ld, state, scale=0.5) for t in range(3)]
    settled()
    check_o(torch.stack(o, 1), ro, sz, dk, 3, dtype, prompt=False)
    check_state(state, rs, sz, 3)


def test_step_touches_its_state_alone_and_without_memory():
    q, k, v, _, state = make(2, 1, 2, 2, 2, 2, 33, 30, F32)
    ld = torch.tensor([-math.inf, 0.0]).cuda()
    buf = torch.full((state.numel() + 64,), 5.0, device="cuda")
    place = buf[32:-32].view_as(state).copy_(state)
    place[:, 0] = 1e30  # forgotten whatever it is
    o = torch.empty(2, 2, 30, device="cuda")
    fm.flash_mca_decay_step(q[:, 0], k[:, 0], v[:, 0], ld, place, o)
    settled()
    assert (buf[:32] == 5).all() and (buf[-32:] == 5).all()
    own = k[:, 0, 0, :, None] * v[:, 0, 0, None, :]
    assert torch.equal(place[:, 0], own)
    ro, rs, sz = serve.decay_attention(q, k, v, [0.0, 0.0], state)
    check_state(place[:, 1], rs[:, 1], {"state": sz["state"][:, 1]}, 1)
    check_o(o[:, None, 1:], ro[:, :, 1:], {"whole": sz["whole"][:, :, 1:]}, 33, 1, F32)


def test_prompt_then_steps_is_the_whole_prompt():
    q, k, v, ld, _ = make(3, 140, 4, 4, 2, 4, 64, 64, BF16)
    n = 130
    _, state = fm.decay_attention(q[:, :n], k[:, :n], v[:, :n], ld, scale=0.125)
    o = [fm.decay_step(q[:, t], k[:, t], v[:, t], ld, state, scale=0.125) for t in range(n, 140)]
    settled()
    ro, rs, sz = serve.decay_attention(q, k, v, ld, None, 0.125)
    sz1 = {key: x[:, n:] for key, x in sz.items() if key != "state"}
    check_o(torch.stack(o, 1), ro[:, n:], sz1, 64, 140, BF16, prompt=False)
    check_state(state, rs, sz, 140)


def test_another_stream_and_refusals():
    q, k, v, ld, state = make(1, 200, 2, 2, 2, 2, 64, 64, BF16)
    want, s = fm.decay_attention(q, k, v, ld, state=state)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, s2 = fm.decay_attention(q, k, v, ld, state=state, stream=side)
    side.synchronize()
    assert torch.equal(o, want) and torch.equal(s, s2)
    with pytest.raises(ValueError):
        fm.decay_attention(q, k[:, :, :, :32], v, ld)
    with pytest.raises(ValueError):
        fm.decay_attention(q, k.float(), v, ld)
    with pytest.raises(ValueError):
        fm.decay_attention(q.transpose(2, 3), k, v, ld)
    with pytest.raises(ValueError):
        fm.decay_attention(q, k, v, ld, state=state[:, :1])
    with pytest.raises(ValueError):
        fm.decay_attention(q, k, v, ld, lengths=torch.tensor([3]).cuda())
    with pytest.raises(ValueError):
        fm.decay_attention(q, k, v, ld.cpu())
    with pytest.raises(TypeError):
        fm.decay_attention(q.half(), k.half(), v.half(), ld)
    for heads in (3, 1):
        with pytest.raises(fm.FmcaError):
            fm.decay_attention(q, k, v, torch.zeros(heads).cuda())
    with pytest.raises(fm.FmcaError):
        fm.decay_step(q[:, 0], k[:, 0], v[:, 0], ld, state, scale=math.nan)
    with pytest.raises(fm.FmcaError):
        fm.decay_attention(q[:, :0], k[:, :0], v[:, :0], ld)
