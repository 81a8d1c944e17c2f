"""CPU oracle of rotary positions and of the paged KV cache (numpy, float64), for
tests only: every row, slot and key on its own, from the definitions."""
from __future__ import annotations

import math

import numpy as np


def frequencies(r, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=None):
    """(radians a position of each pair, factor of cosine and sine)."""
    high = (32.0 if scaling == "yarn" else 4.0) if high is None else high
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    theta, scale = [], 1.0
    for i in range(r // 2):
        t = base ** (-2 * i / r)
        if scaling == "linear":
            t = t / factor
        elif scaling == "yarn":
            d = [r * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (high, low)]
            first, last = max(0, math.floor(d[0])), min(r - 1, math.ceil(d[1]))
            fall = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            t = t * (1 - fall) + t / factor * fall
            scale = 0.1 * math.log(factor) + 1
        elif scaling == "bands":
            turns = original * t / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            t = t * keep + t / factor * (1 - keep)
        theta.append(t)
    return np.array(theta), scale


def positions(start, offsets, depth=None):
    """The position of every row that belongs to a request."""
    out = []
    for b in range(len(start)):
        for t in range(offsets[b], offsets[b + 1]):
            out.append(int(start[b]) + (t - int(offsets[b]) if depth is None else int(depth[t])))
    return np.array(out, dtype=np.int64)


def rotate(x, position, theta, scale=1.0, interleaved=False):
    """x [T][H][D] float64 by its rows' positions.  Returns (y, |x_a| + |x_b| of
    each rotated element's pair, 0 elsewhere)."""
    y, size = x.copy(), np.zeros_like(x)
    r = 2 * len(theta)
    for i, t in enumerate(theta):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        angle = position.astype(np.float64) * t
        c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = scale * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


def place(table, b, slot, page_size):
    return int(table[b][slot // page_size]), slot % page_size


def write(pool, rows, table, prefix, offsets):
    """Rows [T][H][D] into a copy of pool [pages][H][page size][D]."""
    out = pool.copy()
    for b in range(len(prefix)):
        for t in range(offsets[b], offsets[b + 1]):
            page, at = place(table, b, int(prefix[b]) + t - int(offsets[b]), pool.shape[2])
            out[page, :, at] = rows[t]
    return out


def compact(pool, table, prefix, path, accept):
    out = pool.copy()
    for b in range(len(prefix)):
        for j in range(1, int(accept[b]) + 1):
            p0, s0 = place(table, b, int(prefix[b]) + int(path[b][j]), pool.shape[2])
            p1, s1 = place(table, b, int(prefix[b]) + j, pool.shape[2])
            out[p1, :, s1] = pool[p0, :, s0]
    return out


def sees(n, L, parents=None):
    """[n][L + n]: the prefix, and a node's path or (parents None) a token's past."""
    out = np.zeros((n, L + n), dtype=bool)
    out[:, :L] = True
    for i in range(n):
        if parents is None:
            out[i, L:L + i + 1] = True
            continue
        j = i
        while j >= 0:
            out[i, L + j] = True
            j = int(parents[j])
    return out


def attn(q, k_pool, v_pool, table, prefix, offsets, parents=None, scale=None, visible=None, rows=None):
    """Attention in float64.  visible(b): [n][L + n] in place of sees().  Returns (o,
    sum p |v|, largest sum |q||k| scale of a visible key, visible keys) of all rows,
    or of `rows`: what bounds an implementation's rounding."""
    T, Hq, D = q.shape
    H, P = k_pool.shape[1:3]
    G = Hq // H
    scale = 1 / math.sqrt(D) if scale is None else scale
    o, size = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    big, count = np.zeros((T, Hq)), np.zeros(T)
    for b in range(len(prefix)):
        lo, hi, L = int(offsets[b]), int(offsets[b + 1]), int(prefix[b])
        mine = np.arange(lo, hi) if rows is None else np.array([t for t in rows if lo <= t < hi], dtype=int)
        if len(mine) == 0:
            continue
        n = hi - lo
        ok = (visible(b) if visible else sees(n, L, None if parents is None else parents[lo:hi]))[mine - lo]
        slots = np.arange(L + n)
        at = np.asarray(table[b])[slots // P]
        count[mine] = ok.sum(-1)
        for h in range(H):
            k, v = k_pool[at, h, slots % P].astype(np.float64), v_pool[at, h, slots % P].astype(np.float64)
            x = q[mine, h * G:(h + 1) * G].astype(np.float64)
            s = np.where(ok[:, None, :], (x @ k.T) * scale, -np.inf)
            top = s.max(-1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            total = p.sum(-1, keepdims=True)
            p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
            o[mine, h * G:(h + 1) * G] = p @ v
            size[mine, h * G:(h + 1) * G] = p @ np.abs(v)
            big[mine, h * G:(h + 1) * G] = np.where(ok[:, None, :], (np.abs(x) @ np.abs(k).T) * scale, 0).max(-1)
    return o, size, big, count
