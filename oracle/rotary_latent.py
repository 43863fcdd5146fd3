"""Plain NumPy forms of the rotated appends and of latent attention, in
float64.  They share no code with the CUDA path.

The rotation is defined in fp32 arithmetic (each product and each sum
rounded), so that 8-bit codes have one right answer; everything else is
computed in float64.
"""

from __future__ import annotations

import numpy as np

from oracle.pkv_oracle import bf16_to_f64, e4m3_encode, gather, row_scale_exponent


def f64_to_bf16(x):
    """bf16 bit patterns of finite values that fp32 holds exactly (ties to even)."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) & 0xFFFF).astype(np.uint16)


def rotate(x, table_rows, interleaved):
    """x [T, heads, D] float64 with the first R dims rotated by table_rows
    [T, R] (cosines, then sines); every product and sum rounded to fp32.
    Returns float64 values that fp32 holds."""
    f32 = np.float32
    R = table_rows.shape[1]
    half = R // 2
    c = np.asarray(table_rows[:, :half], f32)[:, None, :]
    s = np.asarray(table_rows[:, half:], f32)[:, None, :]
    out = np.array(x, dtype=np.float64, copy=True)
    ia, ib = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, half), slice(half, R))
    a, b = np.asarray(x[..., ia], f32), np.asarray(x[..., ib], f32)
    out[..., ia] = (a * c - b * s).astype(np.float64)
    out[..., ib] = (b * c + a * s).astype(np.float64)
    return out


def rotate_bits(bits, positions, table, interleaved):
    """rotate() of bf16 bit patterns, rounded once to bf16 bit patterns."""
    return f64_to_bf16(rotate(bf16_to_f64(bits), table[positions], interleaved))


def quantize_values(x):
    """E4M3 codes and scale bytes of float64 rows x [..., D]."""
    amax = np.abs(x).max(axis=-1)
    e = np.vectorize(row_scale_exponent, otypes=[np.int64])(amax)
    return e4m3_encode(x * np.exp2(-e.astype(np.float64))[..., None]), (e + 127).astype(np.uint8)


def write_latent(c_new, k_pe, positions, table, slots, cache, interleaved):
    """Latent pages [NB, P, 576] (bits) after the append."""
    out = np.array(cache, copy=True)
    rot = rotate_bits(k_pe[:, None], positions, table, interleaved)[:, 0]
    for t, s in enumerate(np.asarray(slots)):
        if s >= 0:
            out[s // cache.shape[1], s % cache.shape[1]] = np.concatenate([c_new[t], rot[t]])
    return out


def attend_latent(q, cache, block_tables, seq_lens, query_start_loc, scale):
    """(out, bound): attention [T, H, 512] of bf16 bits q [T, H, 576] over
    latent pages, and how far a result may be from it element by element.

    The bound counts the roundings of a bf16 output from bf16 weights and fp32
    sums: the output's half step, 2^-8 |out|; the weights' half steps, to first
    order sum_k w_k 2^-8 |v_k - out| (the row sum adds the rounded weights);
    and the fp32 score, off by at most 576 * 2^-23 of the sum of its terms'
    magnitudes, which moves a weight by that fraction, as exp's own 2^-20."""
    P = cache.shape[1]
    T = q.shape[0]
    out = np.zeros((T, q.shape[1], 512))
    bound = np.zeros_like(out)
    q64 = bf16_to_f64(q)
    for b, L in enumerate(np.asarray(seq_lens)):
        q0, q1 = int(query_start_loc[b]), int(query_start_loc[b + 1])
        if q1 <= q0:
            continue
        rows = gather(cache[:, None], block_tables[b], L, P)[:, 0]
        for t in range(q0, q1):
            n = int(L) - q1 + t + 1
            k, v = rows[:n], rows[:n, :512]
            s = scale * (q64[t] @ k.T)
            w = np.exp(s - s.max(axis=1, keepdims=True))
            w /= w.sum(axis=1, keepdims=True)
            o = w @ v
            terms = scale * (np.abs(q64[t]) @ np.abs(k).T).max(axis=1)
            rel = 2.0 ** -8 + 576 * 2.0 ** -23 * terms + 2.0 ** -20
            spread = w @ np.abs(v) + np.abs(o)
            out[t] = o
            bound[t] = (2.0 ** -8 * np.abs(o) + rel[:, None] * spread) * (1 + 2.0 ** -6) + 1e-30
    return out, bound
