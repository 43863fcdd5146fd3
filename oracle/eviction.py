"""Plain NumPy forms of accumulated attention weights and of eviction by them,
in float64.  They share no code with the CUDA path.

Scores are [NB, Hkv, P] float32: one value a cached token and kv head, in the
place of the token's row in its page.
"""

from __future__ import annotations

import numpy as np


def kept_tokens(scores, L, keep, first, recent):
    """The tokens of one sequence and head that stay, in order, from its L
    scores: the leading `first`, the last `recent` and the largest between
    (ties: the lowest token; NaN as -infinity)."""
    if L <= keep:
        return np.arange(L)
    f = min(first, keep)
    r = min(recent, keep - f)
    with np.errstate(invalid="ignore"):
        middle = np.asarray(scores, dtype=np.float64)[f:L - r]
    middle = np.where(np.isnan(middle), -np.inf, middle)
    best = np.argsort(-middle, kind="stable")[:keep - f - r] + f
    return np.concatenate([np.arange(f), np.sort(best), np.arange(L - r, L)])


def evict(pools, scores, block_tables, seq_lens, keep, first=None, recent=0):
    """([pools], scores, new_lens): the arrays [NB, Hkv, P, ...] of `pools`
    (K, V, scale bytes) and the scores with every sequence cut down."""
    P = scores.shape[2]
    out = [np.array(p, copy=True) for p in pools]
    new_scores = np.array(scores, copy=True)
    lens = np.asarray(seq_lens).copy()
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        m = int(keep[b])
        if L <= m:
            continue
        lens[b] = m
        token = np.arange(L)
        page, row = np.asarray(block_tables[b])[token // P], token % P
        for h in range(scores.shape[1]):
            src = kept_tokens(scores[page, h, row], L, m, 0 if first is None else int(first[b]), recent)
            for new, old in zip(out + [new_scores], list(pools) + [scores]):
                new[page[:m], h, row[:m]] = old[page[src], h, row[src]]
    return out, new_scores, lens
