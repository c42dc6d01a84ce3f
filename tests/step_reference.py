"""Plain references of the step-preparation calls, in whole numbers and in
64-bit floating point, from their definitions in ``include/pa.h``."""

from __future__ import annotations

import math

import numpy as np

import paged_kv_cache_202_gb300 as pa


def step_maps(cache, new, free, count, table, bs, num_blocks, max_seq_len, T):
    """Token by token. Returns (seq, start, pos, slots, table, left, error bits)."""
    cache, new, table = np.asarray(cache), np.asarray(new), np.array(table, dtype=np.int32)
    B, MB = table.shape
    limit = min(max_seq_len, MB * bs)
    err = 0
    if not 0 <= count <= len(free):
        count, err = 0, pa.PA_DEVERR_TABLE
    start, ok, need = [0], [], []
    for b in range(B):
        c, n = int(cache[b]), int(new[b])
        end = start[-1] + max(n, 0)
        good = n >= 0 and c >= 0 and c + n <= limit and end <= T
        if not good:
            err |= pa.PA_DEVERR_SEQ_LEN
        ok.append(good)
        need.append(-(-(c + n) // bs) + (-c // bs) if good else 0)
        start.append(end)
    if sum(need) > count:
        err |= pa.PA_DEVERR_NO_BLOCKS
        ok = [o and not n for o, n in zip(ok, need)]
        need = [0] * B
    pos, slots = np.zeros(T, dtype=np.int32), np.full(T, -1, dtype=np.int64)
    stack = [int(x) for x in free[:count]]
    seq = np.zeros(B, dtype=np.int32)
    for b in range(B):
        if not ok[b]:
            continue
        c, n = int(cache[b]), int(new[b])
        seq[b] = c + n
        had = -(-c // bs)
        for j in range(need[b]):
            table[b, had + j] = stack.pop()
        for i in range(n):
            p = c + i
            phys = int(table[b, p // bs])
            pos[start[b] + i] = p
            if 0 <= phys < num_blocks:
                slots[start[b] + i] = phys * bs + p % bs
            else:
                err |= pa.PA_DEVERR_TABLE
    return (seq, np.minimum(start, T).astype(np.int32), pos, slots, table, len(stack), err)


def inv_freq(rot, base, scaling, factor=1.0, orig=0.0, low=1.0, high=32.0):
    """(frequencies, amplitude) of the scalings, written from their definitions."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if scaling == pa.PA_ROPE_NONE:
        return f, 1.0
    if scaling == pa.PA_ROPE_LINEAR:
        return f / factor, 1.0
    if scaling == pa.PA_ROPE_PARTS:
        turns = orig * f / (2 * math.pi)
        ramp = np.clip((turns - low) / (high - low), 0.0, 1.0)
        return (1 - ramp) * f / factor + ramp * f, 1.0
    at = lambda t: rot * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
    if hi <= lo:
        hi = lo + 0.001
    ramp = np.clip((i - lo) / (hi - lo), 0.0, 1.0)
    return ramp * f / factor + (1 - ramp) * f, 0.1 * math.log(factor) + 1.0


def norm_rope(x, pos, freq, amp, rot, interleaved, weight=None, eps=1e-6):
    """(values, a bound on the 32-bit arithmetic's error) of [T, H, D] rows, 64 bits.

    The bound, in units u = 2^-24 of the pair's magnitude |x1| + |x2| (of |x|
    for an element that is not rotated). Rotation: sine and cosine are off by
    at most 4u (the remainder's conversion u * pi/4, the function's 2 ulp, the
    amplitude's product), each product and the sum round once: 7u; 8u is
    taken. The angle itself is off by |pos| f 2^-51 (the fraction's rounding
    and this reference's own). Norm: the squares of 16 elements a thread are
    summed in a chain and across 8 threads in 3 to 4 more steps, all terms
    positive, so the mean is within 22u, its root within 11u; rsqrt is within
    4u and two products follow: 17u; 20u is taken, before the rotation.
    """
    u = 2.0 ** -24
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    mag_u = 0.0
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
        mag_u = 20.0
    out, bound = y.copy(), mag_u * u * np.abs(y)
    if rot:
        a = np.asarray(pos, dtype=np.float64)[:, None] * freq
        c, s = (amp * np.cos(a))[:, None, :], (amp * np.sin(a))[:, None, :]
        i = np.arange(rot // 2)
        e1, e2 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        x1, x2 = y[..., e1], y[..., e2]
        out[..., e1], out[..., e2] = x1 * c - x2 * s, x2 * c + x1 * s
        m = (np.abs(x1) + np.abs(x2)) * abs(amp)
        far = np.abs(a)[:, None, :] * 2.0 ** -51
        bound[..., e1] = bound[..., e2] = m * ((8.0 + mag_u) * u + far)
    assert out.shape[-1] == D
    return out, bound
