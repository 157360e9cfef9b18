"""Argument checks of generation with states (CPU: every call here is refused before
anything reaches a device)."""
import ctypes

import pytest
import torch

import flash_mixed_chunk_gb300 as fm

BAD = (fm.FMCA_ERR_INVALID_ARG, fm.FMCA_ERR_SHAPE, fm.FMCA_ERR_UNSUPPORTED, fm.FMCA_ERR_ALIGN,
       fm.FMCA_ERR_WORKSPACE)
P = 1 << 20  # a made-up device address, aligned to anything; never read


def shape(B=2, T=64, H=4, Hq=4, Hk=2, Hv=1, dk=16, dv=24, q=None, k=None, v=None):
    s = fm.FmcaDecayShape(B, T, H, Hq, Hk, Hv, dk, dv)
    s.q_stride[:] = q or (T * Hq * dk, Hq * dk, dk)
    s.k_stride[:] = k or (T * Hk * dk, Hk * dk, dk)
    s.v_stride[:] = v or (T * Hv * dv, Hv * dv, dv)
    return s


def attention(s, q=P, k=2 * P, v=3 * P, rate=4 * P, lengths=None, si=5 * P, o=6 * P, so=7 * P,
              scale=1.0, dtype=fm.FMCA_F32, ws=8 * P, ws_bytes=1 << 62):
    return fm.lib.flash_mca_decay_attention(q, k, v, rate, lengths, si, o, so,
                                            ctypes.byref(s) if s else None, scale, dtype, ws,
                                            ws_bytes, None)


def step(s, q=P, k=2 * P, v=3 * P, rate=4 * P, state=5 * P, o=6 * P, scale=1.0,
         dtype=fm.FMCA_F32):
    return fm.lib.flash_mca_decay_step(q, k, v, rate, state, o, ctypes.byref(s), scale, dtype,
                                       None)


def test_workspace_bytes():
    f, none = fm.lib.flash_mca_decay_workspace_bytes, ctypes.c_size_t(-1).value
    for t in (fm.FMCA_F32, fm.FMCA_BF16):
        assert f(ctypes.byref(shape(T=1)), t) == 0
        assert f(ctypes.byref(shape(B=1, T=8192, H=1, Hq=1, Hk=1)), t) % 256 == 0
        assert 0 < f(ctypes.byref(shape(B=1, T=8192, H=1, Hq=1, Hk=1)), t) < 1 << 30
    for s in (shape(B=0), shape(T=0), shape(H=3), shape(dk=257), shape(dv=0), shape(Hk=3),
              shape(q=(-1, 64, 16)), shape(v=(24, 1 << 41, 24)), shape(T=2 ** 31 - 1),
              shape(B=2 ** 31 - 1, H=64, Hq=1, Hk=1)):
        assert f(ctypes.byref(s), fm.FMCA_F32) == none
    assert f(ctypes.byref(shape()), 7) == none and f(None, fm.FMCA_F32) == none


@pytest.mark.parametrize("s, status", [
    (dict(B=0), fm.FMCA_ERR_INVALID_ARG), (dict(T=-1), fm.FMCA_ERR_INVALID_ARG),
    (dict(Hv=0), fm.FMCA_ERR_INVALID_ARG), (dict(Hk=3), fm.FMCA_ERR_SHAPE),
    (dict(Hq=8), fm.FMCA_ERR_SHAPE), (dict(dk=257), fm.FMCA_ERR_UNSUPPORTED),
    (dict(k=(-64, 16, 16)), fm.FMCA_ERR_SHAPE), (dict(k=(1 << 41, 16, 16)), fm.FMCA_ERR_SHAPE),
    (dict(B=2 ** 30, q=(1 << 40, 64, 16)), fm.FMCA_ERR_UNSUPPORTED),
])
def test_sizes_are_refused(s, status):
    assert attention(shape(**s)) == status
    assert step(shape(**{**s, "T": s.get("T", 1)})) == status


def test_attention_is_refused():
    s = shape()
    n = 2 * 4 * 16 * 24 * 4
    for kw, status in [
            (dict(q=0), fm.FMCA_ERR_INVALID_ARG), (dict(rate=0), fm.FMCA_ERR_INVALID_ARG),
            (dict(o=0), fm.FMCA_ERR_INVALID_ARG), (dict(dtype=3), fm.FMCA_ERR_INVALID_ARG),
            (dict(scale=float("nan")), fm.FMCA_ERR_INVALID_ARG),
            (dict(scale=float("inf")), fm.FMCA_ERR_INVALID_ARG),
            (dict(q=P + 2), fm.FMCA_ERR_ALIGN), (dict(rate=P + 2), fm.FMCA_ERR_ALIGN),
            (dict(q=P + 1, dtype=fm.FMCA_BF16), fm.FMCA_ERR_ALIGN),
            (dict(lengths=P + 2), fm.FMCA_ERR_ALIGN), (dict(si=P + 8), fm.FMCA_ERR_ALIGN),
            (dict(so=P + 4), fm.FMCA_ERR_ALIGN),
            (dict(o=P), fm.FMCA_ERR_INVALID_ARG), (dict(so=3 * P), fm.FMCA_ERR_INVALID_ARG),
            (dict(so=6 * P), fm.FMCA_ERR_INVALID_ARG),
            (dict(so=5 * P + n - 16), fm.FMCA_ERR_INVALID_ARG),  # neither state_in nor apart
            (dict(o=5 * P), fm.FMCA_ERR_INVALID_ARG),
            (dict(lengths=6 * P), fm.FMCA_ERR_INVALID_ARG)]:
        assert attention(s, **kw) == status, kw
    assert attention(None) == fm.FMCA_ERR_INVALID_ARG
    # a state of a dv that is no multiple of 4 is aligned to its elements only
    assert attention(shape(dv=25), si=P + 8, q=0) == fm.FMCA_ERR_INVALID_ARG
    long = shape(B=1, T=8192, H=1, Hq=1, Hk=1)
    need = fm.lib.flash_mca_decay_workspace_bytes(ctypes.byref(long), fm.FMCA_F32)
    far = dict(q=1 << 30, k=2 << 30, v=3 << 30, o=4 << 30, ws_bytes=need)
    assert attention(long, **far, ws=None) == fm.FMCA_ERR_WORKSPACE
    assert attention(long, **{**far, "ws_bytes": need - 1}) == fm.FMCA_ERR_WORKSPACE
    assert attention(long, **far, ws=9 * P + 128) == fm.FMCA_ERR_ALIGN
    assert attention(long, **far, ws=4 << 30) == fm.FMCA_ERR_INVALID_ARG
    assert attention(long, **far, ws=7 * P) == fm.FMCA_ERR_INVALID_ARG


def test_step_is_refused():
    s = shape(T=1)
    assert step(shape(T=2)) == fm.FMCA_ERR_SHAPE
    for kw, status in [(dict(state=0), fm.FMCA_ERR_INVALID_ARG),
                       (dict(v=0), fm.FMCA_ERR_INVALID_ARG),
                       (dict(scale=float("nan")), fm.FMCA_ERR_INVALID_ARG),
                       (dict(state=P + 8), fm.FMCA_ERR_ALIGN), (dict(k=P + 1), fm.FMCA_ERR_ALIGN),
                       (dict(state=P), fm.FMCA_ERR_INVALID_ARG),
                       (dict(o=5 * P), fm.FMCA_ERR_INVALID_ARG),
                       (dict(o=4 * P), fm.FMCA_ERR_INVALID_ARG)]:
        assert step(s, **kw) == status, kw


def select(logits=P, row=100, scores=2 * P, finished=None, score=3 * P, parent=4 * P,
           token=5 * P, B=3, K=4, V=100, n=8, pad=0, dtype=fm.FMCA_F32):
    return fm.lib.flash_mca_beam_select(logits, row, scores, finished, score, parent, token, B, K,
                                        V, n, pad, dtype, None)


def test_select_is_refused():
    for kw, status in [
            (dict(B=0), fm.FMCA_ERR_INVALID_ARG), (dict(K=0), fm.FMCA_ERR_INVALID_ARG),
            (dict(V=0), fm.FMCA_ERR_INVALID_ARG), (dict(n=0), fm.FMCA_ERR_INVALID_ARG),
            (dict(K=33), fm.FMCA_ERR_UNSUPPORTED), (dict(n=33), fm.FMCA_ERR_UNSUPPORTED),
            (dict(pad=100), fm.FMCA_ERR_INVALID_ARG), (dict(pad=-1), fm.FMCA_ERR_INVALID_ARG),
            (dict(row=99), fm.FMCA_ERR_SHAPE), (dict(row=-100), fm.FMCA_ERR_SHAPE),
            (dict(B=2 ** 30), fm.FMCA_ERR_UNSUPPORTED), (dict(dtype=2), fm.FMCA_ERR_INVALID_ARG),
            (dict(logits=0), fm.FMCA_ERR_INVALID_ARG), (dict(token=0), fm.FMCA_ERR_INVALID_ARG),
            (dict(logits=P + 2), fm.FMCA_ERR_ALIGN), (dict(scores=P + 2), fm.FMCA_ERR_ALIGN),
            (dict(parent=P + 4), fm.FMCA_ERR_ALIGN), (dict(score=P), fm.FMCA_ERR_INVALID_ARG),
            (dict(parent=5 * P), fm.FMCA_ERR_INVALID_ARG),
            (dict(finished=3 * P), fm.FMCA_ERR_INVALID_ARG)]:
        assert select(**kw) == status, kw


def reorder(*pieces, n=None, parent=1 << 40, B=2, K=4):
    p = (fm.FmcaBeamPiece * max(len(pieces), 1))(*[fm.FmcaBeamPiece(*x) for x in pieces])
    return fm.lib.flash_mca_beam_reorder(p, len(pieces) if n is None else n, parent, B, K, None)


def test_reorder_is_refused():
    good = (P, 64, 64)
    for args, kw, status in [
            ((), {}, fm.FMCA_ERR_INVALID_ARG), ((good,), dict(parent=0), fm.FMCA_ERR_INVALID_ARG),
            ((good,), dict(B=0), fm.FMCA_ERR_INVALID_ARG),
            ((good,), dict(K=33), fm.FMCA_ERR_UNSUPPORTED),
            ((good,), dict(parent=P * 2 + 4), fm.FMCA_ERR_ALIGN),
            (((0, 64, 64),), {}, fm.FMCA_ERR_INVALID_ARG),
            (((P, 63, 64),), {}, fm.FMCA_ERR_SHAPE), (((P, 64, -1),), {}, fm.FMCA_ERR_SHAPE),
            ((good, (P + 500, 64, 64)), {}, fm.FMCA_ERR_INVALID_ARG),
            ((good,), dict(parent=P + 448), fm.FMCA_ERR_INVALID_ARG),
            (((P, 1 << 40, 1 << 40),), dict(B=2 ** 30), fm.FMCA_ERR_UNSUPPORTED)]:
        assert reorder(*args, **kw) == status, (args, kw)
    f = fm.lib.flash_mca_decode_reorder
    need = fm.flash_mca_decode_state_bytes(8, 16, 32, 64, fm.FMCA_BF16)
    ok = [P, need, 1 << 40, 2, 4, 16, 32, 64, 10, fm.FMCA_BF16, None]
    for i, bad, status in [(0, 0, fm.FMCA_ERR_WORKSPACE), (1, need - 1, fm.FMCA_ERR_WORKSPACE),
                           (0, P + 128, fm.FMCA_ERR_ALIGN), (2, 0, fm.FMCA_ERR_INVALID_ARG),
                           (3, 0, fm.FMCA_ERR_INVALID_ARG), (4, 33, fm.FMCA_ERR_WORKSPACE),
                           (5, 300, fm.FMCA_ERR_INVALID_ARG), (8, -1, fm.FMCA_ERR_INVALID_ARG),
                           (9, 5, fm.FMCA_ERR_INVALID_ARG), (2, P, fm.FMCA_ERR_INVALID_ARG),
                           (3, 2 ** 31 - 1, fm.FMCA_ERR_UNSUPPORTED)]:
        args = list(ok)
        args[i] = bad
        assert f(*args) == status, (i, bad)


def test_python_wrappers_refuse_host_tensors():
    q = torch.zeros(1, 4, 2, 8)
    ld, parent = torch.zeros(2), torch.zeros(1, 4, dtype=torch.int64)
    with pytest.raises(ValueError):
        fm.decay_attention(q, q, q, ld)
    with pytest.raises(ValueError):
        fm.flash_mca_decay_attention(q, q, q, ld, None, None, q, None, None)
    with pytest.raises(ValueError):
        fm.decay_step(q[0], q[0], q[0], ld, torch.zeros(4, 2, 8, 8))
    with pytest.raises(ValueError):
        fm.beam_select(torch.zeros(1, 4, 9), torch.zeros(1, 4))
    with pytest.raises(ValueError):
        fm.beam_reorder([torch.zeros(4, 2)], parent)
    with pytest.raises(ValueError):
        fm.flash_mca_decode_reorder(torch.zeros(8, dtype=torch.uint8), parent, 8, 8, 8, 0, 0)
