"""CPU oracle of the 4-bit KV cache (numpy, float64), for tests only.

Every choice the format makes is made here by exhaustive comparison: the
scale of a group is the one whose sixfold is nearest to the group's largest
magnitude, a code the one whose value times the scale is nearest to the
element; ties go to the even byte or code.  All those products and
differences are exact in float64: of float32 magnitudes (24 bits) cut to the
largest value of the table they are compared with (which keeps the nearest),
where the table's steps are no finer than 2^-18.
"""
from __future__ import annotations

import numpy as np

GROUP = 16
MAX_SCALE_BYTE = 226
CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def record_bytes(D: int) -> int:
    return -(-(D + D // 8) // 16) * 16


def scale_value(byte):
    byte = np.asarray(byte, dtype=np.int64)
    e, m = byte >> 3, byte & 7
    return np.where(e == 0, m * 2.0 ** -17, (1 + m / 8) * np.exp2(e - 15.0))


SCALES = scale_value(np.arange(MAX_SCALE_BYTE + 1))


def _nearest(x, table):
    """Index of the table entry nearest to x >= 0 (ties: the even index)."""
    x = np.minimum(x, table[-1])
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    d = (x - table[lo]) - (table[hi] - x)          # exact: > 0 when the upper one is nearer
    return np.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)


def quantise(x):
    """Codes (one per element) and scale bytes (one per 16) of rows [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], g, 0.0)
    byte = _nearest(np.abs(g).max(-1), 6 * SCALES)
    s = SCALES[byte][..., None]
    code = np.zeros(g.shape, dtype=np.int64)
    best = np.full(g.shape, np.inf)
    for i in (0, 2, 4, 6, 1, 3, 5, 7):             # even codes first: they keep a tie
        d = np.abs(np.minimum(np.abs(g), 6 * s) - CODES[i] * s)
        code, best = np.where(d < best, i, code), np.minimum(d, best)
    code = np.where(s == 0, 0, code) | np.where(np.signbit(g), 8, 0)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8), finite


def records(k, v):
    """Records [..., R] of rows k, v [..., D]."""
    D = k.shape[-1]
    out = np.zeros(k.shape[:-1] + (record_bytes(D),), dtype=np.uint8)
    for i, x in enumerate((k, v)):
        code, byte, _ = quantise(x)
        out[..., i * D // 2:(i + 1) * D // 2] = code[..., 0::2] | code[..., 1::2] << 4
        out[..., D + i * D // 16:D + (i + 1) * D // 16] = byte
    return out


def values(rec, D):
    """Keys and values (float64) of records [..., R]."""
    out = []
    for i in range(2):
        b = rec[..., i * D // 2:(i + 1) * D // 2]
        c = np.stack([b & 15, b >> 4], -1).reshape(b.shape[:-1] + (D,))
        x = CODES[c & 7] * np.where(c >= 8, -1.0, 1.0)
        out.append(x * np.repeat(scale_value(rec[..., D + i * D // 16:D + (i + 1) * D // 16]), GROUP, axis=-1))
    return out


def write(cache, k, v, start, offsets):
    """spec_kv4_write on a numpy cache, in place (no errors)."""
    for b in range(len(start)):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        cache[b, :, start[b]:start[b] + hi - lo] = records(k[lo:hi], v[lo:hi]).transpose(1, 0, 2)


def read(cache, D, start, offsets):
    parts = [cache[b, :, start[b]:start[b] + offsets[b + 1] - offsets[b]].transpose(1, 0, 2) for b in range(len(start))]
    return values(np.concatenate(parts), D)


def sees(parents, L, window=0, sinks=0):
    """[n][L + n]: the keys each node of one tree sees."""
    n = len(parents)
    out = np.zeros((n, L + n), dtype=bool)
    depth = np.zeros(n, dtype=np.int64)
    for i in range(n):
        depth[i] = 0 if i == 0 else depth[parents[i]] + 1
        out[i, :L] = True
        j = i
        while j >= 0:
            out[i, L + j] = True
            j = int(parents[j])
        if window > 0:
            at = np.concatenate([np.arange(L), L + depth[:n]])
            out[i] &= (at > L + depth[i] - window) | (at < sinks)
    return out


def tree_attn(q, cache, prefix_lens, offsets, parents, window=0, sinks=0, scale=None):
    """Attention in float64.  Returns (o, mean |v|, largest sum |q||k| scale of a
    visible key, sum of the visible |v|): the last three ([T][Hq][D], [T][Hq] and
    [T][Hq][D]) bound an implementation's rounding."""
    T, Hq, D = q.shape
    B, H = cache.shape[:2]
    G = Hq // H
    scale = 1 / np.sqrt(D) if scale is None else scale
    o, size, big = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    reach = np.zeros((T, Hq, D))
    for b in range(B):
        lo, hi, L = int(offsets[b]), int(offsets[b + 1]), int(prefix_lens[b])
        ok = sees(parents[lo:hi], L, window, sinks)
        for h in range(H):
            k, v = values(cache[b, h, :L + hi - lo], D)
            x = q[lo:hi, h * G:(h + 1) * G].astype(np.float64)
            s = np.where(ok[:, None, :], np.einsum("ngd,sd->ngs", x, k) * scale, -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o[lo:hi, h * G:(h + 1) * G] = np.einsum("ngs,sd->ngd", p, v)
            size[lo:hi, h * G:(h + 1) * G] = np.einsum("ngs,sd->ngd", p, np.abs(v))
            reach[lo:hi, h * G:(h + 1) * G] = (ok.astype(np.float64) @ np.abs(v))[:, None]
            part = np.einsum("ngd,sd->ngs", np.abs(x), np.abs(k)) * scale
            big[lo:hi, h * G:(h + 1) * G] = np.where(ok[:, None, :], part, 0).max(-1)
    return o, size, big, reach
