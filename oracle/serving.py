"""fp64 definitions of the rotary positions and of the paged-cache operators,
one element after the other (CPU, test infrastructure; shares nothing with the
CUDA path)."""

from __future__ import annotations

import math

import numpy as np


def rope(x, pos, inv_freq, axis, layout, inverse=False):
    """x [B, S, H, D], pos [n_axes, B, S]: pairs turned by pos[axis[p]] * inv_freq[p]."""
    y = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    for p in range(n):
        if not 0 <= axis[p] < pos.shape[0]:
            continue
        i, j = (2 * p, 2 * p + 1) if layout == "interleaved" else (p, p + n)
        f = float(inv_freq[p]) if math.isfinite(inv_freq[p]) else 0.0
        ang = pos[axis[p]].astype(np.float64) * f
        c, s = np.cos(ang)[:, :, None], np.sin(ang)[:, :, None] * (-1.0 if inverse else 1.0)
        a, b = np.array(y[..., i]), np.array(y[..., j])
        y[..., i], y[..., j] = a * c - b * s, a * s + b * c
    return y


def _seen(word, length, n_new):
    """The slots a token sees, from its tree word (None: all of the new tokens up to itself are in it)."""
    return list(range(length)) + [length + j for j in range(n_new) if (int(word) >> j) & 1]


def words_or_chain(tree, B, T):
    if tree is None:
        return [[(1 << (t + 1)) - 1 for t in range(T)] for _ in range(B)]
    return [[int(w) & ((1 << 64) - 1) for w in row] for row in tree]


def attend(q, seq_k, seq_v, length, n_new, words, scale):
    """q [B, T, H, D]; seq_k[b], seq_v[b] [slots, H_kv, D]: (O, LSE [B, H, T],
    sum_j p_j |v_j| (the weight a relative error of p carries into O))."""
    B, T, H, D = q.shape
    O, mass = np.zeros((B, T, H, D)), np.zeros((B, T, H, D))
    L = np.full((B, H, T), -np.inf)
    for b in range(B):
        G = H // seq_k[b].shape[1]
        for t in range(min(T, n_new[b])):
            j = _seen(words[b][t], length[b], n_new[b])
            if not j:
                continue
            for h in range(H):
                s = scale * (seq_k[b][j, h // G] @ q[b, t, h])
                m = s.max()
                e = np.exp(s - m)
                O[b, t, h] = e @ seq_v[b][j, h // G] / e.sum()
                mass[b, t, h] = e @ np.abs(seq_v[b][j, h // G]) / e.sum()
                L[b, h, t] = m + np.log(e.sum())
    return O, L, mass


def weigh(scores, q, seq_k, lse, length, n_new, words, scale):
    """scores [B, H_kv, capacity] plus each slot's attention weight."""
    out = np.array(scores, dtype=np.float64)
    B, T, H, _ = q.shape
    for b in range(B):
        G = H // seq_k[b].shape[1]
        for t in range(min(T, n_new[b])):
            j = _seen(words[b][t], length[b], n_new[b])
            for h in range(H):
                if j and np.isfinite(lse[b, h, t]):
                    out[b, h // G, j] += np.exp(scale * (seq_k[b][j, h // G] @ q[b, t, h]) - lse[b, h, t])
    return out


def evict_sources(score, pos, n, budget, sinks, recent, next_pos):
    """Which old slot each kept slot [0, min(n, budget)) takes its key from."""
    if n <= budget:
        return list(range(n))

    def rank(i):
        must = pos[i] < sinks or pos[i] >= next_pos - recent
        s = -math.inf if math.isnan(score[i]) else float(score[i])
        return (not must, 0.0 if must else -s, not must and math.isnan(score[i]), i)

    kept = set(sorted(range(n), key=rank)[:budget])
    movers = iter(sorted(i for i in kept if i >= budget))
    return [i if i in kept else next(movers) for i in range(budget)]
