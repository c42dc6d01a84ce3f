"""Sliding-window attention with sinks in 64-bit floating point, row by row
from its definition, with a bound on the kernels' arithmetic error."""

from __future__ import annotations

import numpy as np


def tokens_seen(p: int, window: int, sinks: int) -> np.ndarray:
    """The tokens t <= p with p - t < window or t < sinks."""
    t = np.arange(p + 1)
    return t[(p - t < window) | (t < sinks)]


def attend(q, k_pool, v_pool, table, p, scale, window, sinks):
    """One query row ([Hq, D]) at position p of the sequence with this table.

    Returns (out, sum_t w_t |v_t|, the largest sum_d |q_d k_td| * |scale| over
    the tokens seen), each per head, 64 bits.
    """
    Hq, D = q.shape
    Hkv, bs = k_pool.shape[1], k_pool.shape[2]
    t = tokens_seen(p, window, sinks)
    blk = table[t // bs]
    assert (blk >= 0).all()
    k, v = (x[blk, :, t % bs].astype(np.float64) for x in (k_pool, v_pool))   # [n, Hkv, D]
    qg = q.astype(np.float64).reshape(Hkv, Hq // Hkv, D)
    s = np.einsum("hgd,nhd->hgn", qg, k) * scale
    mag = (np.einsum("hgd,nhd->hgn", np.abs(qg), np.abs(k)) * abs(scale)).max(-1)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    out = np.einsum("hgn,nhd->hgd", w, v)
    wv = np.einsum("hgn,nhd->hgd", w, np.abs(v))
    return out.reshape(Hq, D), wv.reshape(Hq, D), mag.reshape(Hq, 1)


def tolerance(out, wv, mag, D, p_bits, out_bf16):
    """How far a kernel's row may be from `out`.

    A score is a sum of D exact bf16 products kept in 32 bits, whatever the
    order and with truncation at worst: off by at most D 2^-23 of the sum of
    their magnitudes, which changes each weight by that factor and the
    normalised weight by twice that. Each weight enters the value sum rounded
    to p_bits significant bits (half a step: 2^-p_bits of it) but the row sum
    unrounded; the exponential (2^-22), the rescalings and the sums in 32 bits
    stay within 2^-14 of the weights. The stored value rounds once.
    """
    weights = 2 * D * 2.0 ** -23 * mag + 2.0 ** -p_bits + 2.0 ** -14
    step = 2.0 ** -8 if out_bf16 else 2.0 ** -24
    return weights * wv * (1 + step) + step * np.abs(out) + 1e-30
