"""Plain NumPy forms of accumulated attention weights and of eviction by them,
in float64.  They share no code with the CUDA path.

Scores are [NB, Hkv, P] float32: one value a cached token and kv head, in the
place of the token's row in its page.
"""

from __future__ import annotations

import numpy as np

from oracle.pkv_oracle import bf16_to_f64, gather, gather_fp8


def weigh(q, k_cache, scores, block_tables, seq_lens, query_start_loc, scale, decay=1.0, first=None, scored=None,
          k_scale=None):
    """(scores, bound): float64 scores [NB, Hkv, P] after the attention weights
    of bf16 query bits q [T, Hq, 128] were added, and how far an fp32 result
    may be from them, element by element (0 where nothing was written).

    The bound counts, to first order with room for the second, the roundings
    of fp32 arithmetic: a score s is off by at most 128 * 2^-23 of the sum of
    its terms' magnitudes (a tensor core may truncate where fp32 would round),
    the row's log-sum by as much again; the exponent's argument is rounded
    three times at its size, on both sides; exp2 is off by 2^-21; row sums add
    L terms and token sums n * G, each addition off by 2^-24 of what it has so
    far; the new score is rounded twice."""
    P = k_cache.shape[2]
    Hkv, Hq = k_cache.shape[1], q.shape[1]
    G = Hq // Hkv
    out = np.asarray(scores, dtype=np.float64).copy()
    bound = np.zeros_like(out)
    q64 = bf16_to_f64(q)
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        q0, q1 = int(query_start_loc[b]), int(query_start_loc[b + 1])
        n = q1 - q0
        if n == 0:
            continue
        f = 0 if first is None else max(0, int(first[b]))
        new = L - n if scored is None else int(scored[b])
        keys = gather(k_cache, block_tables[b], L, P) if k_scale is None else \
            gather_fp8(k_cache, k_scale, block_tables[b], L, P)
        token = np.arange(L)
        page, row = np.asarray(block_tables[b])[token // P], token % P
        for g in range(Hkv):
            rows = q64[q0:q1, g * G:(g + 1) * G].reshape(n * G, -1)
            s = scale * (rows @ keys[:, g].T)
            s = np.where(token[None] <= (L - n + np.arange(n * G) // G)[:, None], s, -np.inf)
            w = np.exp(s - s.max(axis=1, keepdims=True))
            w /= w.sum(axis=1, keepdims=True)
            total = w.sum(axis=0)
            terms = scale * (np.abs(rows) @ np.abs(keys[:, g]).T).max()
            size = np.abs(s[np.isfinite(s)]).max() / np.log(2.0)
            rel = 2 * 128 * 2.0 ** -23 * terms + 6 * 2.0 ** -24 * size + 2.0 ** -20 + (L + n * G) * 2.0 ** -24
            with np.errstate(invalid="ignore"):
                old = np.where(token < new, decay * out[page, g, row] if decay else 0.0, 0.0)
            on = token >= f
            out[page[on], g, row[on]] = (old + total)[on]
            bound[page[on], g, row[on]] = (1.01 * rel * total + 2.0 ** -22 * np.abs(old) + 1e-36)[on]
    return out, bound


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
