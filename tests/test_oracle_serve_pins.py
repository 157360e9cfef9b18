"""Pins of the oracle of generation with states (CPU): the token recurrence against the
whole weight matrix, worked examples, the selection against a sort of all candidates."""
import math

import numpy as np
import pytest

from oracle import serve


def test_two_tokens_by_hand():
    # lam = 1/2, one head, dk = 2, dv = 1
    q = np.array([[[[1.0, 2.0]], [[3.0, -1.0]]]])
    k = np.array([[[[2.0, 0.0]], [[1.0, 1.0]]]])
    v = np.array([[[[4.0]], [[-2.0]]]])
    s0 = np.array([[[[1.0], [3.0]]]])
    # S1 = (1/2, 3/2) + (8, 0) = (8.5, 1.5);  o1 = 8.5 + 3 = 11.5
    # S2 = (4.25, 0.75) + (-2, -2) = (2.25, -1.25);  o2 = 6.75 + 1.25 = 8
    o, s, _ = serve.decay_attention(q, k, v, [math.log(0.5)], s0)
    assert np.allclose(o.ravel(), [11.5, 8.0]) and np.allclose(s.ravel(), [2.25, -1.25])
    o, s, _ = serve.decay_attention(q, k, v, [math.log(0.5)], s0, scale=2.0, lengths=[1])
    assert np.allclose(o.ravel(), [23.0, 0.0]) and np.allclose(s.ravel(), [8.5, 1.5])
    o, s, _ = serve.decay_attention(q, k, v, [math.log(0.5)], s0, lengths=[0])
    assert not o.any() and np.array_equal(s, s0)


@pytest.mark.parametrize("H,Hq,Hk,Hv", [(1, 1, 1, 1), (4, 2, 1, 4), (6, 3, 6, 2)])
def test_recurrence_is_the_weight_matrix(H, Hq, Hk, Hv):
    rng = np.random.default_rng(H)
    B, T, dk, dv = 2, 150, 3, 5
    q, k = rng.normal(size=(B, T, Hq, dk)), rng.normal(size=(B, T, Hk, dk))
    v, s0 = rng.normal(size=(B, T, Hv, dv)), rng.normal(size=(B, H, dk, dv))
    ld = -rng.uniform(0.001, 1.0, size=H)
    o, s, size = serve.decay_attention(q, k, v, ld, s0, scale=0.7)
    gap = np.arange(T)[:, None] - np.arange(T)[None, :]
    for b in range(B):
        for h in range(H):
            x, y, z = q[b, :, h * Hq // H], k[b, :, h * Hk // H], v[b, :, h * Hv // H]
            w = np.where(gap >= 0, np.exp(ld[h] * np.maximum(gap, 0)), 0.0)
            far = np.exp(ld[h] * (np.arange(T) + 1))[:, None] * (x @ s0[b, h])
            assert np.allclose(o[b, :, h], 0.7 * ((x @ y.T * w) @ z + far))
            assert np.allclose(s[b, h], np.exp(ld[h] * T) * s0[b, h] +
                               (y * np.exp(ld[h] * (T - 1 - np.arange(T)))[:, None]).T @ z)
    # the sums of absolute values bound what they stand for
    assert (np.abs(o) <= size["near"] + size["far"] + 1e-12).all()
    assert (size["near"] <= size["whole"] + 1e-12).all()
    assert (np.abs(s) <= size["state"] + 1e-12).all()


def test_pieces_of_a_sequence_and_no_memory():
    rng = np.random.default_rng(1)
    q, k, v = (rng.normal(size=(1, 9, 2, 4)) for _ in range(3))
    ld = np.array([-0.3, -math.inf])
    o, s, _ = serve.decay_attention(q, k, v, ld)
    o1, s1, _ = serve.decay_attention(q[:, :4], k[:, :4], v[:, :4], ld)
    o2, s2, _ = serve.decay_attention(q[:, 4:], k[:, 4:], v[:, 4:], ld, s1)
    assert np.allclose(o, np.concatenate([o1, o2], 1)) and np.allclose(s, s2)
    # the head without memory sees its own token alone
    own = np.einsum("btd,btd->bt", q[:, :, 1], k[:, :, 1])[..., None] * v[:, :, 1]
    assert np.allclose(o[:, :, 1], own)


def test_selection_by_hand():
    z = np.log(np.array([[[1.0, 2.0, 1.0], [3.0, 3.0, 6.0]]]))  # p: 1/4 1/2 1/4 | 1/4 1/4 1/2
    s = np.log(np.array([[0.5, 0.25]]))
    # 1/8 1/4 1/8 | 1/16 1/16 1/8
    score, parent, token = serve.beam_select(z, s, 4)
    assert np.allclose(np.exp(score), [[0.25, 0.125, 0.125, 0.125]])
    assert parent.tolist() == [[0, 0, 0, 1]] and token.tolist() == [[1, 0, 2, 2]]
    # the second beam finished: itself with the pad token, ahead of 1/8
    score, parent, token = serve.beam_select(z, s, 3, finished=[[False, True]], pad=2)
    assert np.allclose(np.exp(score), [[0.25, 0.25, 0.125]])
    assert parent.tolist() == [[0, 1, 0]] and token.tolist() == [[1, 2, 0]]


def test_selection_without_candidates():
    z = np.array([[[0.0, -np.inf], [np.nan, 0.0], [np.inf, 0.0], [-np.inf, -np.inf],
                   [0.0, 0.0]]])
    s = np.array([[0.0, 0.0, 0.0, 0.0, -np.inf]])
    score, parent, token = serve.beam_select(z, s, 7, pad=1)
    assert score[0, 0] == 0.0 and np.isneginf(score[0, 1:]).all()
    assert parent.tolist() == [[0, 1, 2, 3, 4, 0, 1]] and token.tolist() == [[0] + [1] * 6]


@pytest.mark.parametrize("K,V,n", [(1, 7, 3), (3, 11, 6), (4, 40, 32)])
def test_selection_is_a_sort_of_all(K, V, n):
    rng = np.random.default_rng(V)
    z = np.round(rng.normal(size=(5, K, V)) * 4) / 4  # many ties
    s = -rng.integers(0, 3, size=(5, K)).astype(float)
    score, parent, token = serve.beam_select(z, s, n)
    p = np.exp(z) / np.exp(z).sum(2, keepdims=True)
    c = s[..., None] + np.log(p)
    for b in range(5):
        flat = np.round(c[b].ravel(), 12)
        at = np.argsort(-flat, kind="stable")[:n]
        m = len(at)
        assert np.allclose(score[b, :m], flat[at])
        # equal sums may round apart in the last place: compare the values' order there
        assert np.allclose(flat[parent[b, :m] * V + token[b, :m]], flat[at])


def test_reorder_rows():
    rows = np.arange(6)[:, None] * np.ones((1, 2))
    got = serve.reorder(rows, [[1, 1, 0], [2, 5, -1]])
    assert got[:, 0].tolist() == [1, 1, 0, 5, 4, 5]
