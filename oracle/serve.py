"""fp64 oracle of generation with states: linear attention with a decay for each
head, beam search's selection, and the reordering of rows by their parents.

Plain numpy in the definitions' order (a token at a time, a candidate at a time);
shares no code with the CUDA library.  Test infrastructure only.
"""
from __future__ import annotations

import math

import numpy as np


def _f64(x):
    return np.asarray(x.detach().cpu().double().numpy() if hasattr(x, "detach") else x,
                      dtype=np.float64)


def _to_heads(x, H):
    """[..., heads, d] with a head for each of H."""
    return np.repeat(x, H // x.shape[-2], axis=-2)


def decay_attention(q, k, v, log_decay, state=None, scale=1.0, lengths=None):
    """S_t = exp(log_decay) S_{t-1} + k_t^T v_t, o_t = scale q_t S_t, a token at a time.

    Returns (o [B, T, H, dv], state [B, H, dk, dv], size): `size` holds, for the
    bounds of rounding errors, the same sums over absolute values: "near" and "far"
    [B, T, H, dv] (what a token's chunk of 128 and what lies before it add to an
    output, with |q k| as it is), "whole" (with |q| |k|), "state"."""
    q, k, v, ld = _f64(q), _f64(k), _f64(v), _f64(log_decay)
    B, T = q.shape[:2]
    H = ld.shape[0]
    q, k, v = _to_heads(q, H), _to_heads(k, H), _to_heads(v, H)
    dk, dv = q.shape[-1], v.shape[-1]
    lam = np.exp(ld)[:, None, None]
    o = np.zeros((B, T, H, dv))
    near, far, whole = np.zeros_like(o), np.zeros_like(o), np.zeros_like(o)
    out, size = np.zeros((B, H, dk, dv)), np.zeros((B, H, dk, dv))
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        S = np.zeros((H, dk, dv)) if state is None else _f64(state)[b].copy()
        A = np.abs(S)
        start = S
        for t in range(n):
            c = t // 128 * 128
            if t == c:
                start = S.copy()
            S = lam * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            A = lam * A + np.abs(k[b, t])[:, :, None] * np.abs(v[b, t])[:, None, :]
            o[b, t] = scale * np.einsum("hd,hdv->hv", q[b, t], S)
            whole[b, t] = abs(scale) * np.einsum("hd,hdv->hv", np.abs(q[b, t]), A)
            gap = np.arange(t - c, -1, -1)
            with np.errstate(invalid="ignore"):
                w = np.where(gap[:, None] == 0, 1.0, np.exp(gap[:, None] * ld[None]))
                ahead = np.exp((t - c + 1) * ld)[:, None]
            p = np.abs(np.einsum("hd,jhd->jh", q[b, t], k[b, c:t + 1])) * w
            near[b, t] = abs(scale) * np.einsum("jh,jhv->hv", p, np.abs(v[b, c:t + 1]))
            far[b, t] = abs(scale) * ahead * np.einsum("hd,hdv->hv", np.abs(q[b, t]),
                                                       np.abs(start))
        out[b], size[b] = S, A
    return o, out, {"near": near, "far": far, "whole": whole, "state": size}


def beam_select(logits, scores, n, finished=None, pad=0):
    """(score [B, n], parent, token) of the n largest candidates, equal ones by the
    lowest parent * V + token."""
    logits, scores = _f64(logits), _f64(scores)
    B, K = scores.shape
    logits = logits.reshape(B, K, -1)
    V = logits.shape[2]
    score = np.full((B, n), -np.inf)
    parent = np.tile(np.arange(n) % K, (B, 1))
    token = np.full((B, n), pad)
    for b in range(B):
        found = []
        for k in range(K):
            s, z = scores[b, k], logits[b, k]
            if not math.isfinite(s):
                continue
            if finished is not None and bool(finished[b][k]):
                found.append((-s, k * V + pad))
                continue
            top = z.max()  # NaN where there is one
            if not math.isfinite(top):
                continue
            lse = top + math.log(np.exp(z - top).sum())
            best = np.argsort(-z, kind="stable")[:n]
            found += [(-(s + (z[v] - lse)), k * V + v) for v in best if z[v] > -np.inf]
        for i, (c, at) in enumerate(sorted(found)[:n]):
            score[b, i], parent[b, i], token[b, i] = -c, at // V, at % V
    return score, parent, token


def reorder(rows, parent):
    """rows [B K, ...] -> row (b, k) is what row (b, parent[b, k]) was."""
    rows, parent = np.asarray(rows), np.asarray(parent)
    B, K = parent.shape
    out = rows.copy()
    for b in range(B):
        for k in range(K):
            p = parent[b, k]
            if 0 <= p < K:
                out[b * K + k] = rows[b * K + p]
    return out
