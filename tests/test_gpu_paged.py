"""Rotary positions and the paged KV cache on the GPU against a float64 oracle.
Copies are exact; rotation and attention are held to bounds counted from the
roundings they make."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import token_tree_verification_gb300 as ttv
from oracle import paged

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
LAYOUTS = pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def zeros_status(B):
    return torch.zeros(B, dtype=torch.int32, device="cuda")


def f64(x):
    return x.double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gpu(x, dtype):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def bits(x):
    return x.view(torch.int16 if x.dtype == BF16 else torch.int32)


def random_tree(rng, n, chain=False):
    return [-1] + [i - 1 if chain else int(rng.integers(max(0, i - 10), i)) for i in range(1, n)]


def depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def strided(rng, T, H, D, dtype, spare=0, shift=0):
    """Rows [T][H][D] inside a wider row of H + spare heads, `shift` elements from a 16-byte boundary."""
    width = (H + spare) * D + (8 if shift else 0)
    base = gpu(rng.standard_normal((T, width)), dtype)
    return base.as_strided((T, H, D), (width, D, 1), shift)


# ------------------------------------------------------------------ rotary positions
def assert_rotated(y, x, position, theta, scale, interleaved):
    ref, size = paged.rotate(f64(x), position, theta, scale, interleaved)
    # cosine and sine: one ulp of each (2^-24 at most), the half turns' rounding to
    # 2^-25 (times pi), the table's double; two products and a sum in fp32; scale
    # and its product.  Together below 2^-20 of |x_a| + |x_b|; then the result's half step
    bound = 2.0 ** -20 * size + half_step(y.dtype) * np.abs(ref) + 2.0 ** -133
    err = np.abs(f64(y) - ref)
    assert (err <= bound).all(), (err - bound).max()


@DTYPES
@LAYOUTS
@pytest.mark.parametrize("D,r,H,spare,shift", [(128, 128, 5, 0, 0), (128, 64, 3, 2, 0), (64, 64, 1, 0, 0), (64, 16, 9, 4, 0),
                                               (128, 24, 2, 0, 0), (128, 6, 2, 1, 3), (96, 96, 3, 0, 0), (8, 2, 1, 0, 0),
                                               (512, 512, 2, 0, 0), (136, 80, 3, 0, 1)])
def test_rope_on_ragged_rows(gpu_lib, dtype, interleaved, D, r, H, spare, shift):
    rng = np.random.default_rng(D + r + H)
    n = [3, 0, 37, 1, 0, 64]
    off = np.concatenate([[0], np.cumsum(n)])
    T = int(off[-1])
    start = [0, 5, 1000, 8191, 3, 70000]
    theta, scale = paged.frequencies(r, 10000.0)
    table = ttv.rope_table(r, 10000.0)
    x = strided(rng, T + 4, H, D, dtype, spare, shift)
    out = torch.full((T + 4, H, D), 7.0, dtype=dtype, device="cuda")
    status = zeros_status(len(n))
    y = ttv.rope(x, table, i32(start), i32(off), status, interleaved=interleaved, out=out)
    assert y is out and status.eq(0).all()
    assert out[T:].eq(7.0).all()                       # rows behind the last request
    assert_rotated(out[:T], x[:T], paged.positions(start, off), theta, scale, interleaved)
    assert torch.equal(out[:T, :, r:], x[:T, :, r:])   # the other dims are copied
    # in place, into the same strided rows, gives the same bits
    ttv.rope(x, table, i32(start), i32(off), status, interleaved=interleaved, out=x)
    assert torch.equal(bits(x[:T].contiguous()), bits(out[:T]))


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0), ("bands", 8.0)])
def test_rope_for_long_contexts(gpu_lib, scaling, factor):
    rng = np.random.default_rng(5)
    theta, scale = paged.frequencies(128, 10000.0, scaling, factor, 4096.0)
    table = ttv.rope_table(128, 10000.0, scaling, factor, original=4096.0)
    off, start = [0, 40, 50], [100, 131072]
    x = gpu(rng.standard_normal((50, 2, 128)), F32)
    y = ttv.rope(x, table, i32(start), i32(off), zeros_status(2))
    assert_rotated(y, x, paged.positions(start, off), theta, scale, False)


def test_rope_far_away(gpu_lib):
    """A position of 2^31 - 2: the angle of an exact product, modulo whole turns."""
    x = torch.ones((2, 1, 8), dtype=F32, device="cuda")
    table = ttv.rope_table(8, 10.0)
    y = ttv.rope(x, table, i32([2 ** 31 - 2]), i32([0, 2]), zeros_status(1))
    for t in range(2):
        for i in range(4):
            # whole turns leave the 64-bit product by themselves; Python's integers keep it all
            turns = (2 ** 31 - 2 + t) * table.freqs[i].item() % 2 ** 64 / 2 ** 64
            c, s = math.cos(2 * math.pi * turns), math.sin(2 * math.pi * turns)
            assert abs(y[t, 0, i].item() - (c - s)) <= 2.0 ** -19
            assert abs(y[t, 0, i + 4].item() - (c + s)) <= 2.0 ** -19


@LAYOUTS
def test_rope_far_away_by_the_formula(gpu_lib, interleaved):
    """Positions up to 2^31 + 6 against angles of 60 digits, without the table."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")
    x = torch.zeros((3, 1, 128), dtype=F32, device="cuda")
    x[:, :, 0::2 if interleaved else 1] = 1.0
    if not interleaved:
        x[:, :, 64:] = 0.0
    start, depth = 2 ** 31 - 3, [0, 2, 9]
    y = ttv.rope(x, ttv.rope_table(128, 500000.0), i32([start]), i32([0, 3]), zeros_status(1), depth=i32(depth),
                 interleaved=interleaved)[:, 0].double().cpu().numpy()
    for t in range(3):
        for i in range(64):
            turns = (start + depth[t]) * Decimal(500000) ** (Decimal(-2 * i) / 128) / (2 * pi)
            angle = 2 * math.pi * float(turns % 1)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 64)
            # half turns rounded to 2^-25 (times pi), the turn's lower bits cut (2^-32), the table's half unit 2^31
            # times over; an ulp of cosine and sine (2^-24); times one and plus zero are exact
            bound = math.pi * 2.0 ** -25 + 2 * math.pi * (2.0 ** -32 + 2.0 ** -34) + 2.0 ** -24
            assert abs(y[t, a] - math.cos(angle)) <= bound and abs(y[t, b] - math.sin(angle)) <= bound, (t, i)


def test_rope_of_trees_and_of_many_requests(gpu_lib):
    rng = np.random.default_rng(9)
    B = 1500
    n = rng.integers(0, 6, B)
    n[777] = 500
    off = np.concatenate([[0], np.cumsum(n)])
    depth = np.concatenate([depths(random_tree(rng, k)) if k else [] for k in n]).astype(int)
    start = rng.integers(0, 5000, B)
    theta, scale = paged.frequencies(64)
    x = gpu(rng.standard_normal((off[-1], 2, 64)), BF16)
    status = zeros_status(B)
    y = ttv.rope(x, ttv.rope_table(64), i32(start), i32(off), status, depth=i32(depth))
    assert status.eq(0).all()
    assert_rotated(y, x, paged.positions(start, off, depth), theta, scale, False)


@pytest.mark.parametrize("T", [1, 4, 2500, 20000])
def test_rope_at_every_launch_shape(gpu_lib, T):
    rng = np.random.default_rng(T)
    theta, scale = paged.frequencies(128)
    x = gpu(rng.standard_normal((T, 10, 128)), BF16)
    y = ttv.rope(x, ttv.rope_table(128), i32([17]), i32([0, T]), zeros_status(1))
    assert_rotated(y, x, paged.positions([17], [0, T]), theta, scale, False)


@DTYPES
@LAYOUTS
@pytest.mark.parametrize("D,r,shift", [(128, 24, 0), (80, 20, 0), (64, 36, 0), (72, 18, 0), (128, 64, 4), (128, 64, 2), (96, 8, 6), (64, 64, 5)])
@pytest.mark.parametrize("T", [9, 3000])
def test_rope_in_narrow_pieces(gpu_lib, dtype, interleaved, D, r, shift, T):
    """Pairs' ends and rows that do not start on 16 bytes."""
    rng = np.random.default_rng(D + r + shift)
    H, off = 24, [0, 2, 2, T]
    start = [3, 0, 100]
    theta, scale = paged.frequencies(r)
    x = strided(rng, T, H, D, dtype, 1, shift)
    y = ttv.rope(x, ttv.rope_table(r), i32(start), i32(off), zeros_status(3), interleaved=interleaved)
    assert_rotated(y, x, paged.positions(start, off), theta, scale, interleaved)
    assert torch.equal(y[:, :, r:], x[:, :, r:])
    # on the way into pages, keys and values at other alignments than the queries'
    k, v = strided(rng, T, 2, D, dtype, 0, 0), strided(rng, T, 2, D, dtype, 1, shift)
    cache, status = Cache(rng, [T + 3, 1, T + 100], 2, 64, D, dtype, fill=5.0), zeros_status(3)
    q_out = ttv.rope_write_paged(x, k, v, cache.k, cache.v, cache.block_table, i32(start), i32(off), status, ttv.rope_table(r),
                                 interleaved=interleaved)
    assert status.eq(0).all() and torch.equal(bits(q_out), bits(y))
    turned = ttv.rope(k, ttv.rope_table(r), i32(start), i32(off), status, interleaved=interleaved)
    for pool, rows in ((cache.k, turned), (cache.v, v)):
        want = paged.write(np.full(pool.shape, 5.0), f64(rows), cache.table, start, off)
        assert (f64(pool) == want).all()


def test_rope_errors_leave_rows_alone(gpu_lib):
    table = ttv.rope_table(64)
    x = torch.randn((12, 2, 64), device="cuda")
    good = ttv.rope(x, table, i32([0, 5, 9]), i32([0, 4, 8, 12]), zeros_status(3))
    out = torch.full_like(x, 3.0)
    status = zeros_status(3)
    ttv.rope(x, table, i32([0, -5, 9]), i32([0, 4, 8, 12]), status, out=out)
    assert status.tolist() == [0, -10, 0]
    assert torch.equal(out[:4], good[:4]) and out[4:8].eq(3).all() and torch.equal(out[8:], good[8:])
    for off, want in (([0, 4, 13, 12], [0, -4, -4]), ([0, 8, 4, 12], [0, -4, 0]), ([-1, 4, 8, 12], [-4, 0, 0])):
        status = zeros_status(3)
        ttv.rope(x, table, i32([0, 0, 0]), i32(off), status, out=torch.empty_like(x))
        assert status.tolist() == want, off
    status, out = zeros_status(1), torch.full_like(x, 3.0)
    depth = [0, 1, 2, -1] + list(range(8))
    ttv.rope(x, table, i32([0]), i32([0, 12]), status, depth=i32(depth), out=out)
    assert status.tolist() == [-10] and out[3].eq(3).all() and not out[2].eq(3).any()


# ------------------------------------------------------------------ pages
class Cache:
    """A pool and block table of requests with the given slots, pages in no order, -1 behind the last."""

    def __init__(self, rng, slots, H, P, D, dtype, spare=3, fill=math.nan):
        need = [-(-s // P) for s in slots]
        self.total = sum(need) + spare
        order = rng.permutation(self.total)
        self.table = np.full((len(slots), max(max(need), 1)), -1)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.P = P
        self.k, self.v = (torch.full((self.total, H, P, D), fill, dtype=dtype, device="cuda") for _ in range(2))

    def fill(self, rng, slots, size=1.0):
        """Random keys and values in the slots in use; the others stay as they are (NaN)."""
        for b, s in enumerate(slots):
            for i in range(-(-s // self.P)):
                m = min(self.P, s - i * self.P)
                for x in (self.k, self.v):
                    x[self.table[b, i], :, :m] = gpu(size * rng.standard_normal((x.shape[1], m, x.shape[3])), x.dtype)
        return self

    @property
    def block_table(self):
        return i32(self.table)


@DTYPES
@LAYOUTS
@pytest.mark.parametrize("P,D,r,Hq,Hkv,spare,tree", [(16, 128, 128, 8, 2, 1, False), (8, 64, 32, 3, 3, 0, True),
                                                     (64, 128, 24, 4, 1, 2, True), (256, 64, 64, 2, 2, 0, False),
                                                     (4096, 128, 0, 1, 1, 0, False)])
def test_rows_into_pages(gpu_lib, dtype, interleaved, P, D, r, Hq, Hkv, spare, tree):
    rng = np.random.default_rng(P + D + r)
    n = [17, 1, 40, 5] if tree else [33, 0, 130, 1]
    L = [P - 1, 0, 3 * P + 5, 70]
    off = np.concatenate([[0], np.cumsum(n)])
    T = int(off[-1])
    depth = np.concatenate([depths(random_tree(rng, k)) for k in n]) if tree else None
    cache = Cache(rng, [a + b for a, b in zip(L, n)], Hkv, P, D, dtype, fill=5.0)
    both = strided(rng, T + 2, Hq + 2 * Hkv, D, dtype, spare)
    q, k, v = both[:, :Hq], both[:, Hq:Hq + Hkv], both[:, Hq + Hkv:]
    table = ttv.rope_table(r) if r else None
    theta, scale = paged.frequencies(r) if r else (np.zeros(0), 1.0)
    q_out = torch.full((T + 2, Hq, D), 7.0, dtype=dtype, device="cuda")
    status = zeros_status(len(n))
    got = ttv.rope_write_paged(q, k, v, cache.k, cache.v, cache.block_table, i32(L), i32(off), status, table,
                               depth=None if depth is None else i32(np.concatenate([depth, [-1, -1]])),
                               interleaved=interleaved, q_out=q_out)
    assert got is q_out and status.eq(0).all() and q_out[T:].eq(7).all()
    position = paged.positions(L, off, depth)
    assert_rotated(q_out[:T], q[:T], position, theta, scale, interleaved)
    want_v = paged.write(np.full(tuple(cache.v.shape), 5.0), f64(v), cache.table, L, off)
    assert (f64(cache.v) == want_v).all()
    # the rotated keys have the bits that spec_rope gives them; no other slot changed
    turned = ttv.rope(k[:T], table or ttv.RopeTable(torch.zeros(0, dtype=torch.int64, device="cuda"), 1.0, 0), i32(L),
                      i32(off), status, depth=None if depth is None else i32(depth), interleaved=interleaved)
    want_k = paged.write(np.full(tuple(cache.k.shape), 5.0), f64(turned), cache.table, L, off)
    assert (f64(cache.k) == want_k).all()
    # keys and values alone, positions of their own
    start = [x + 100 for x in L]
    assert ttv.rope_write_paged(None, k, v, cache.k, cache.v, cache.block_table, i32(L), i32(off), status, table,
                                start=i32(start), interleaved=interleaved) is None
    turned = ttv.rope(k[:T], table or ttv.RopeTable(torch.zeros(0, dtype=torch.int64, device="cuda"), 1.0, 0),
                      i32(start), i32(off), status, interleaved=interleaved)
    assert (f64(cache.k) == paged.write(want_k, f64(turned), cache.table, L, off)).all()
    assert status.eq(0).all()


def test_rows_into_pages_errors(gpu_lib):
    rng = np.random.default_rng(1)
    n, L, P, D = [20, 20, 20], [5, 5, 5], 16, 64
    off = [0, 20, 40, 60]
    q, k, v = (torch.randn((60, h, D), device="cuda") for h in (4, 2, 2))
    rope = ttv.rope_table(64)

    def call(change=None, lens=L, offsets=off):
        cache = Cache(np.random.default_rng(2), [25, 25, 25], 2, P, D, F32, fill=5.0)
        if change:
            change(cache.table)
        out, status = torch.full_like(q, 7.0), zeros_status(3)
        ttv.rope_write_paged(q, k, v, cache.k, cache.v, cache.block_table, i32(lens), i32(offsets), status, rope, q_out=out)
        return status.tolist(), out, cache

    _, good, kept = call()
    for bad in (-1, 9, 2 ** 31 - 1, -2 ** 31):
        def change(t):
            t[1, 1] = bad
        status, out, cache = call(change)
        assert status == [0, -14, 0]
        assert torch.equal(out[:20], good[:20]) and out[20:40].eq(7).all() and torch.equal(out[40:], good[40:])
        mine = kept.table[1]
        assert cache.k[mine].eq(5).all() and cache.v[mine].eq(5).all()
        for b in (0, 2):
            assert torch.equal(cache.k[kept.table[b]], kept.k[kept.table[b]])
    assert call(lens=[5, 13, 5])[0] == [0, -10, 0]        # 33 slots of 32
    assert call(lens=[5, -1, 5])[0] == [0, -10, 0]
    assert call(offsets=[0, 61, 40, 60])[0] == [-4, -4, 0]
    status, out, cache = call(lens=[5, 12, 5])            # the last slot of the last page
    assert status == [0, 0, 0]


@pytest.mark.parametrize("n", [[3000, 40], [4, 3, 5, 1, 8, 2], [70, 1, 600]])
def test_every_page_of_a_run_is_looked_at(gpu_lib, n):
    """A page that is not there, anywhere in a run, keeps every row of the run from being written; a wrong
    depth beside it changes nothing."""
    rng = np.random.default_rng(sum(n))
    P, D, B = 8, 64, len(n)
    L = [3] * B
    off = np.concatenate([[0], np.cumsum(n)])
    T = int(off[-1])
    q, k, v = (torch.randn((T, h, D), device="cuda") for h in (2, 1, 1))
    rope = ttv.rope_table(64)
    depth = np.concatenate([np.arange(m) for m in n])
    kept = Cache(rng, [a + b for a, b in zip(n, L)], 1, P, D, F32, fill=5.0)

    def call(table, depth):
        cache = [torch.full_like(kept.k, 5.0) for _ in range(2)]
        out, status = torch.full_like(q, 7.0), zeros_status(B)
        ttv.rope_write_paged(q, k, v, *cache, i32(table), i32(L), i32(off), status, rope, depth=i32(depth), q_out=out)
        return status.tolist(), out, cache

    status, good, written = call(kept.table, depth)
    assert status == [0] * B
    for b in range(B):
        last = (n[b] + L[b] - 1) // P
        for page in sorted({0, last, last // 2, last // 3, max(0, last - 1)}):
            for row in (None, 0, n[b] // 2, n[b] - 1):
                table, deep = kept.table.copy(), depth.copy()
                table[b, page] = -1 if page % 2 else kept.total
                if row is not None:
                    deep[off[b] + row] = -1
                status, out, cache = call(table, deep)
                assert status[b] in ((-14,) if row is None else (-14, -10)) and sum(map(bool, status)) == 1
                assert out[off[b]:off[b + 1]].eq(7).all()
                for x, y in zip(cache, written):
                    mine = torch.from_numpy(kept.table[b][:last + 1]).cuda()
                    assert x[mine].eq(5).all()
                    for other in set(range(B)) - {b}:
                        theirs = torch.from_numpy(kept.table[other][kept.table[other] >= 0]).cuda()
                        assert torch.equal(x[theirs], y[theirs])


# ------------------------------------------------------------------ attention
def attn_bound(o, size, big, count, D, dtype):
    """Scores: D products summed in fp32, the scale; weights: the exponential's
    argument and value, for bf16 the two parts' 2^-17; sums over the keys."""
    u = 2.0 ** -24
    weight = 2 * u * (2 * D + 8) * big[:, :, None] + 8 * u + (2.0 ** -16 if dtype == BF16 else 0)
    total = weight + 2 * u * (count[:, None, None] + 64)
    return half_step(dtype) * np.abs(o) + 2 * total * size + 1e-37


def check_attn(got, q, cache, L, off, parents=None, scale=None, visible=None, rows=None):
    o, size, big, count = paged.attn(f64(q), f64(cache.k), f64(cache.v), cache.table, L, off, parents, scale, visible, rows)
    rows = np.arange(int(off[-1])) if rows is None else np.array(rows)
    err = np.abs(f64(got)[rows] - o[rows])
    bound = attn_bound(o, size, big, count, q.shape[2], q.dtype)[rows]
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(~(err <= bound))[:4].tolist())


def batch(rng, n, L, Hq, Hkv, P, D, dtype, size=1.0, extra=0):
    off = np.concatenate([[0], np.cumsum(n)])
    cache = Cache(rng, [a + b for a, b in zip(n, L)], Hkv, P, D, dtype).fill(rng, [a + b for a, b in zip(n, L)], size)
    q = gpu(size * rng.standard_normal((int(off[-1]) + extra, Hq, D)), dtype)
    return q, cache, off


@DTYPES
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,P,n,L", [
    (4, 4, 16, [8], [128]), (3, 1, 16, [1, 128, 37], [0, 0, 1]), (8, 1, 64, [5, 64], [700, 63]), (2, 2, 8, [128], [500]),
    (5, 1, 32, [128, 1, 30], [127, 128, 129]), (16, 2, 128, [1, 1, 1, 1, 1], [0, 1, 127, 128, 1000]),
    (1, 1, 256, [2], [2050]), (128, 1, 16, [3, 1], [40, 300]), (2, 1, 4096, [17], [4090]), (12, 4, 64, [100, 128], [5, 260])])
def test_trees(gpu_lib, dtype, D, Hq, Hkv, P, n, L):
    rng = np.random.default_rng(Hq * 1000 + P + sum(n) + sum(L))
    q, cache, off = batch(rng, n, L, Hq, Hkv, P, D, dtype, extra=3)
    parents = np.concatenate([random_tree(rng, k) for k in n])
    status = zeros_status(len(n))
    T = int(off[-1])
    padded = i32(np.concatenate([parents, [-1] * 3]))
    mask, _ = ttv.build_tree_mask(padded[:T].contiguous(), i32(off), status)
    mask = torch.cat([mask, mask[:1].expand(3, 4)])
    o = torch.full_like(q, 7.0)
    args = (q, cache.k, cache.v, cache.block_table, i32(L), i32(off))
    assert ttv.tree_attn_paged(*args, mask, max(L), status, o=o) is o
    assert status.eq(0).all() and o[T:].eq(7).all()
    check_attn(o, q, cache, L, off, parents)
    # by the parents, with another bound on the prefixes (another number of splits)
    p = torch.full_like(q, 7.0)
    ttv.tree_attn_paged(*args, None, max(L) + 5000, status, o=p, parents=padded)
    assert status.eq(0).all() and p[T:].eq(7).all()
    check_attn(p, q, cache, L, off, parents)


@DTYPES
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,P,n,L", [
    (4, 4, 16, [129], [0]), (3, 1, 16, [0, 300, 0, 1], [9, 0, 0, 500]), (8, 1, 64, [65, 64, 63, 200], [700, 0, 1, 64]),
    (2, 2, 8, [513], [37]), (6, 2, 128, [1, 128, 256], [127, 128, 129]), (1, 1, 32, [700], [1300]), (40, 1, 64, [90], [130])])
def test_chunks(gpu_lib, dtype, D, Hq, Hkv, P, n, L):
    rng = np.random.default_rng(Hq * 1000 + P + sum(n) + sum(L))
    q, cache, off = batch(rng, n, L, Hq, Hkv, P, D, dtype, extra=2)
    status = zeros_status(len(n))
    o = torch.full_like(q, 7.0)
    ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, max(L), status, o=o, causal=True)
    assert status.eq(0).all() and o[int(off[-1]):].eq(7).all()
    check_attn(o, q, cache, L, off)


@pytest.mark.parametrize("n,L,Hq,Hkv,P,causal", [([2000], [9000], 8, 1, 64, True), ([6, 6, 6], [20000, 11000, 3], 4, 4, 16, False),
                                                 ([1] * 40, list(range(0, 4000, 100)), 16, 2, 32, False),
                                                 ([3000, 1, 700], [0, 12000, 4096], 4, 2, 128, True)])
def test_long_ones_on_a_sample_of_rows(gpu_lib, n, L, Hq, Hkv, P, causal):
    rng = np.random.default_rng(sum(n))
    q, cache, off = batch(rng, n, L, Hq, Hkv, P, 128, BF16)
    T = int(off[-1])
    parents = np.concatenate([random_tree(rng, k, chain=True) for k in n])
    status = zeros_status(len(n))
    o = ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, max(L), status,
                            parents=None if causal else i32(parents), causal=causal)
    assert status.eq(0).all()
    rows = sorted({0, T - 1, T // 2} | set(rng.integers(0, T, 40).tolist()))
    check_attn(o, q, cache, L, off, None, rows=rows)


def test_many_requests_among_them_empty_ones(gpu_lib):
    rng = np.random.default_rng(3)
    B = 300
    n, L = rng.integers(0, 9, B), rng.integers(0, 70, B)
    n[210] = 400
    q, cache, off = batch(rng, n.tolist(), L.tolist(), 4, 2, 16, 64, BF16)
    status = zeros_status(B)
    o = ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, 70, status, causal=True)
    assert status.eq(0).all()
    check_attn(o, q, cache, L, off)


@DTYPES
@pytest.mark.parametrize("B,causal", [(64, False), (65, False), (65, True), (1100, False), (1100, True)])
def test_hundreds_of_requests(gpu_lib, dtype, B, causal):
    """Runs that fill blocks of rows exactly (32 x 4), end inside one or are empty; some are wrong."""
    rng = np.random.default_rng(B + causal)
    n = rng.choice([0, 1, 4, 5, 32, 33] if causal else [1, 4, 5, 32, 33], B)
    n[[0, 7, B - 1]] = 96, 128, 32
    L = rng.integers(0, 40, B)
    q, cache, off = batch(rng, n.tolist(), L.tolist(), 4, 1, 8, 64, dtype, extra=200)
    parents = np.concatenate([random_tree(rng, k) for k in n] + [np.full(200, -1)])
    T, wrong_page, wrong_prefix = int(off[-1]), 7, B - 2
    table, lens = cache.table.copy(), L.copy()
    table[wrong_page, -(-(n[7] + L[7]) // 8) - 1] = cache.total
    lens[wrong_prefix] = -1
    for split in (70, 100000):
        status, o = zeros_status(B), torch.full_like(q, 7.0)
        ttv.tree_attn_paged(q, cache.k, cache.v, i32(table), i32(lens), i32(off), None, split, status, o=o, causal=causal,
                            parents=None if causal else i32(parents))
        assert np.flatnonzero(status.cpu().numpy()).tolist() == [wrong_page, wrong_prefix]
        assert status[wrong_page] == -14 and status[wrong_prefix] == -10
        left = np.zeros(T + 200, dtype=bool)
        left[T:] = True
        for b in (wrong_page, wrong_prefix):
            left[off[b]:off[b + 1]] = True
        assert o[torch.from_numpy(left).cuda()].eq(7).all()
        check_attn(o, q, cache, L, off, None if causal else parents, rows=np.flatnonzero(~left[:T]))


@DTYPES
@pytest.mark.parametrize("wrong", [-2 ** 31, -1, 2 ** 31 - 1, 10 ** 6])
@pytest.mark.parametrize("B", [3, 70, 600])
def test_offsets_that_are_anything(gpu_lib, dtype, wrong, B):
    """The request behind a wrong offset and the one before it report it; others are right or left out."""
    rng = np.random.default_rng(B)
    n, L = [3] * B, [20] * B
    q, cache, off = batch(rng, n, L, 16, 1, 16, 64, dtype)
    args = (q, cache.k, cache.v, cache.block_table, i32(L))
    good, status = torch.full_like(q, 7.0), zeros_status(B)
    ttv.tree_attn_paged(*args, i32(off), None, 20, status, o=good, causal=True)
    assert status.eq(0).all()
    for at in sorted({0, 1, B // 2, B}):
        bad = off.copy()
        bad[at] = wrong
        o, status = torch.full_like(q, 7.0), zeros_status(B)
        ttv.tree_attn_paged(*args, i32(bad), None, 20, status, o=o, causal=True)
        codes = status.cpu().numpy()
        assert set(np.flatnonzero(codes).tolist()) == {b for b in (at - 1, at) if 0 <= b < B} and set(codes[codes != 0]) == {-4}
        same = (bits(o) == bits(good)).flatten(1).all(1) | (o == 7).flatten(1).all(1)
        assert same.all()
        left = (o == 7).flatten(1).all(1).cpu().numpy()
        for b in (at - 1, at):
            if 0 <= b < B:
                assert left[off[b]:off[b + 1]].all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", ["mask", "parents", "causal"])
def test_many_requests_behind_few_keys(gpu_lib, form, D):
    """More blocks of rows than SMs, a few tiles of keys each."""
    rng = np.random.default_rng(D + len(form))
    B, causal = 150, form == "causal"
    n = rng.choice([0, 1, 40, 130] if causal else [1, 2, 31, 64, 70], B)
    L = rng.choice([0, 1, 63, 64, 127, 128, 129, 200, 383, 512], B)
    q, cache, off = batch(rng, n.tolist(), L.tolist(), 16, 8, 16, D, BF16, extra=5)
    T = int(off[-1])
    parents = None if causal else np.concatenate([random_tree(rng, k) for k in n] + [[-1] * 5])
    status, o, mask = zeros_status(B), torch.full_like(q, 7.0), None
    if form == "mask":
        mask = ttv.build_tree_mask(i32(parents[:T]), i32(off), status)[0]
        mask = torch.cat([mask, mask[:1].expand(5, 4)])
    ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), mask, 512, status, o=o, causal=causal,
                        parents=i32(parents) if form == "parents" else None)
    assert status.eq(0).all() and o[T:].eq(7).all()
    check_attn(o, q, cache, L, off, parents)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [0.01, 6.0, 40.0])
def test_scores_of_every_size_of_many_requests(gpu_lib, size, D):
    rng = np.random.default_rng(5)
    B = 160
    n, L = [2] * B, rng.integers(300, 500, B).tolist()
    q, cache, off = batch(rng, n, L, 8, 8, 64, D, BF16, size=size)
    status = zeros_status(B)
    o = ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, 500, status, causal=True)
    assert status.eq(0).all()
    check_attn(o, q, cache, L, off)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L,Hq,Hkv,P,causal", [
    ([1] * 3, [5000, 0, 4097], 4, 1, 8, True), ([1, 1], [9000, 1], 2, 2, 16, False), ([1] * 70, list(range(0, 700, 10)), 8, 2, 32, True),
    ([8], [2047], 3, 3, 64, False), ([2, 0, 1, 3], [300, 5, 31, 32], 5, 1, 8, True), ([16, 1], [1000, 3], 8, 1, 128, False),
    ([33, 2, 128], [100, 64, 200], 2, 1, 16, False), ([300], [700], 6, 2, 16, True), ([3] * 90, [90] * 90, 1, 1, 4096, False)])
def test_fp32_rows_from_one_to_many(gpu_lib, n, L, Hq, Hkv, P, causal, D):
    rng = np.random.default_rng(sum(n) + sum(L) + D)
    q, cache, off = batch(rng, n, L, Hq, Hkv, P, D, F32, extra=4)
    T, B = int(off[-1]), len(n)
    parents = None if causal else np.concatenate([random_tree(rng, k) for k in n] + [[-1] * 4])
    status, o = zeros_status(B), torch.full_like(q, 7.0)
    ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, max(L), status, o=o, causal=causal,
                        parents=None if causal else i32(parents))
    assert status.eq(0).all() and o[T:].eq(7).all()
    check_attn(o, q, cache, L, off, parents)


def test_calls_of_both_kinds_in_turn(gpu_lib):
    """Launches for many requests and for one long one, and the dense call, each of which may begin while the
    one before it ends; on two streams, captured and not."""
    rng = np.random.default_rng(6)
    B, D, H = 150, 128, 8
    n, L = [2] * B, rng.integers(50, 300, B).tolist()
    many = batch(rng, n, L, H, H, 16, D, BF16)
    one = batch(rng, [64], [1500], H, H, 16, D, BF16)
    parents = i32(random_tree(rng, 64))
    dense = [torch.randn((1, H, 600, D), device="cuda").to(BF16) for _ in range(2)]
    lens, offs, s1, s2 = i32(L), i32(many[2]), zeros_status(B), zeros_status(1)
    tables = many[1].block_table, one[1].block_table
    other = i32([1500]), i32([0, 64]), i32([500])

    def calls():
        out = []
        for _ in range(3):
            out.append(ttv.tree_attn_paged(many[0], many[1].k, many[1].v, tables[0], lens, offs, None, 300, s1, causal=True))
            out.append(ttv.tree_attn_paged(one[0], one[1].k, one[1].v, tables[1], other[0], other[1], None, 1500, s2,
                                           parents=parents))
            out.append(ttv.tree_attn(one[0], *dense, other[2], other[1], None, 500, s2, parents=parents))
            out.append(ttv.tree_attn_paged(many[0], many[1].k, many[1].v, tables[0], lens, offs, None, 300, s1, causal=True))
        return out

    want = calls()
    check_attn(want[0], many[0], many[1], L, many[2])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        with torch.cuda.stream(side):
            beside = calls()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, beside, captured):
            assert torch.equal(a, b) and torch.equal(a, c)
    assert s1.eq(0).all() and s2.eq(0).all()


@DTYPES
def test_scores_of_every_size(gpu_lib, dtype):
    """Scores that rise along the keys by far more than a reference's slack, negative ones,
    and ones beyond 2^31 whose largest alone keeps a weight."""
    rng = np.random.default_rng(4)
    for size in (0.01, 6.0, 40.0):
        q, cache, off = batch(rng, [5, 90], [600, 33], 4, 2, 16, 128, dtype, size=size)
        status = zeros_status(2)
        o = ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32([600, 33]), i32(off), None, 600, status, causal=True)
        check_attn(o, q, cache, [600, 33], off)
    for size in (2.0 ** 14, 2.0 ** 20, 2.0 ** 40):
        # one key on the queries' own line: its score is size^2 / sqrt(D) above the others', exactly
        n, L, D = [3], [500], 64
        q, cache, off = batch(rng, n, L, 1, 1, 16, D, dtype)
        q.fill_(0)
        cache.k[cache.table[0].tolist()] = 0
        q[:, 0, 5] = size
        for slot, sign in ((130, 1.0), (20, -1.0), (400, 2.0), (401, -2.0)):
            page, at = paged.place(cache.table, 0, slot, 16)
            cache.k[page, 0, at, 5] = sign * size
        status = zeros_status(1)
        o = ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, 500, status, causal=True)
        page, at = paged.place(cache.table, 0, 400, 16)
        assert torch.equal(o, cache.v[page, 0, at].expand(3, 1, D)), size


@DTYPES
def test_rows_that_see_nothing_and_values_out_of_range(gpu_lib, dtype):
    rng = np.random.default_rng(6)
    n, L = [4, 130 % 128 + 1], [0, 0]
    q, cache, off = batch(rng, n, L, 2, 2, 8, 64, dtype)
    T = int(off[-1])
    mask = torch.zeros((T, 4), dtype=torch.int32, device="cuda")
    mask[1, 0] = 2                 # node 1 sees itself, node 3 the root, the others nothing
    mask[3, 0] = 1
    mask[2, 3] = -1                # bits behind the tree's nodes are no keys
    status = zeros_status(2)
    o = ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), mask, 0, status)
    assert status.eq(0).all()
    page = cache.table[0, 0]
    assert o[0].eq(0).all() and o[2].eq(0).all() and o[4:].eq(0).all()
    assert torch.equal(o[1], cache.v[page, :, 1]) and torch.equal(o[3], cache.v[page, :, 0])
    # the type's largest and smallest, infinities in a masked place, NaN in one query
    n, L = [8], [40]
    q, cache, off = batch(rng, n, L, 2, 2, 8, 64, dtype)
    clean = ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, 40, status[:1], causal=True)
    page, at = paged.place(cache.table, 0, 47, 8)
    cache.k[page, :, at] = math.inf
    q2 = q.clone()
    q2[2, 1] = math.nan
    o = ttv.tree_attn_paged(q2, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, 40, status[:1], causal=True)
    keep = [(t, h) for t in range(7) for h in range(2) if (t, h) != (2, 1)]
    for t, h in keep:
        assert torch.equal(o[t, h], clean[t, h]), (t, h)
    assert o[2, 1].isnan().all()


def test_pages_give_what_a_dense_cache_gives(gpu_lib):
    rng = np.random.default_rng(8)
    B, n, L, H, D, P = 3, [64, 20, 128], [300, 1, 64], 2, 128, 32
    q, cache, off = batch(rng, n, L, 8, H, P, D, BF16)
    parents = i32(np.concatenate([random_tree(rng, k) for k in n]))
    S = 448
    kd, vd = (torch.zeros((B, H, S, D), dtype=BF16, device="cuda") for _ in range(2))
    for b in range(B):
        used = cache.table[b][:-(-(L[b] + n[b]) // P)].tolist()
        for dense, pool in ((kd, cache.k), (vd, cache.v)):
            dense[b, :, :len(used) * P] = pool[used].transpose(0, 1).flatten(1, 2)
    status = zeros_status(B)
    dense = ttv.tree_attn(q, kd, vd, i32(L), i32(off), None, max(L), status, parents=parents)
    o = ttv.tree_attn_paged(q, cache.k, cache.v, cache.block_table, i32(L), i32(off), None, max(L), status, parents=parents)
    assert status.eq(0).all()
    # each is within a half step and 2^-15 or so of the exact value
    assert ((o.double() - dense.double()).abs() <= 2 * half_step(BF16) * dense.double().abs() + 2e-4).all()


@DTYPES
def test_attention_errors_leave_rows_alone(gpu_lib, dtype):
    rng = np.random.default_rng(11)
    n, L = [30, 40, 20], [200, 100, 300]
    q, cache, off = batch(rng, n, L, 4, 2, 16, 64, dtype)
    parents = i32(np.concatenate([random_tree(rng, k) for k in n]))

    def call(table=None, lens=L, offsets=off, causal=False, par=parents):
        o, status = torch.full_like(q, 7.0), zeros_status(3)
        ttv.tree_attn_paged(q, cache.k, cache.v, i32(cache.table if table is None else table), i32(lens), i32(offsets), None,
                            max(L), status, o=o, parents=None if causal else par, causal=causal)
        return status.tolist(), o

    for causal in (False, True):
        good_status, good = call(causal=causal)
        assert good_status == [0, 0, 0]
        for page, bad in ((0, cache.total), (3, -1), (8, 2 ** 31 - 1)):
            table = cache.table.copy()
            table[1, page] = bad
            status, o = call(table, causal=causal)
            assert status == [0, -14, 0]
            assert torch.equal(o[:30], good[:30]) and o[30:70].eq(7).all() and torch.equal(o[70:], good[70:])
        for lens in ([200, -1, 300], [200, 400, 300], [200, 2 ** 31 - 1, 300]):
            status, o = call(lens=lens, causal=causal)
            assert status == [0, -10, 0] and o[30:70].eq(7).all() and torch.equal(o[70:], good[70:])
        status, o = call(offsets=[0, 30, 91, 90], causal=causal)
        assert status == [0, -4, -4] and o[30:].eq(7).all()
    status, o = call(offsets=[0, 30, 30, 90])             # a tree without nodes
    assert status[1] == -4 and torch.equal(o[:30], call()[1][:30])
    wrong = parents.clone()
    wrong[30 + 5] = 5
    assert call(par=wrong)[0] == [0, -5, 0]


# ------------------------------------------------------------------ moving the accepted path
@DTYPES
@pytest.mark.parametrize("P,D,H", [(8, 64, 1), (16, 128, 3), (64, 128, 2), (4096, 64, 1)])
def test_compaction(gpu_lib, dtype, P, D, H):
    rng = np.random.default_rng(P)
    n, L = [64, 1, 128, 9, 128, 20], [7, 30, 3, 0, P - 1, 11]
    off = np.concatenate([[0], np.cumsum(n)])
    # a path in place, a root alone, every node, the last node, every second, one whose places are later sources
    paths = [list(range(9)), [0], list(range(128)), [0, 8], list(range(0, 128, 2)), [0, 2, 3, 4, 19]]
    W = 128
    path = np.array([p + [-1] * (W - len(p)) for p in paths])
    accept = [len(p) - 1 for p in paths]
    cache = Cache(rng, [a + b for a, b in zip(n, L)], H, P, D, dtype).fill(rng, [a + b for a, b in zip(n, L)])
    want = [paged.compact(f64(x), cache.table, L, path, accept) for x in (cache.k, cache.v)]
    status = zeros_status(len(n))
    lens = ttv.kv_compact_paged(cache.k, cache.v, cache.block_table, i32(L), i32(off), i32(path), i32(accept), status)
    assert status.eq(0).all() and lens.tolist() == [a + 1 + b for a, b in zip(L, accept)]
    for x, y in zip((cache.k, cache.v), want):
        assert np.array_equal(f64(x), y, equal_nan=True)


def test_compaction_errors_leave_the_cache_alone(gpu_lib):
    rng = np.random.default_rng(12)
    n, L = [10] * 8, [20] * 8
    off = np.concatenate([[0], np.cumsum(n)])
    cache = Cache(rng, [30] * 8, 2, 8, 64, F32).fill(rng, [30] * 8)
    path = np.array([[0, 2, 5, -1]] * 8)
    accept, lens, table = [2] * 8, list(L), cache.table.copy()
    path[1, 2] = 2                  # not increasing
    path[2, 2] = 10                 # outside the tree
    path[3, 0] = 1                  # no root
    accept[4] = 4                   # longer than its row
    lens[5] = 2 ** 31 - 3
    table[6, 3] = cache.total       # the page of slot 25, which moves
    status = zeros_status(8)
    status[7] = -5                  # found by another call
    before = [cache.k.clone(), cache.v.clone()]
    got = ttv.kv_compact_paged(cache.k, cache.v, i32(table), i32(lens), i32(off), i32(path), i32(accept), status)
    assert status.tolist() == [0, -5, -5, -5, -4, -10, -14, -5]
    assert got.tolist() == [23] + lens[1:]
    for b in range(1, 8):
        for x, y in zip((cache.k, cache.v), before):
            assert torch.equal(bits(x[cache.table[b].tolist()]), bits(y[cache.table[b].tolist()])), b


@DTYPES
@pytest.mark.parametrize("bad", [[0, -2 ** 31, -2 ** 31 + 1, 3], [0, -2, -1, 3], [0, 2 ** 31 - 1, -5, -4], [-1, 0, 1, 2],
                                 [0, 1, 1, 2], [0, 0, 1, 2], [-2 ** 31, -2 ** 31 + 1, -9, -8], [2 ** 31 - 1] * 4])
def test_compaction_of_paths_that_are_anything(gpu_lib, dtype, bad):
    """Entries that increase from below zero: each looks like a node behind its neighbour, its slot lies far outside."""
    rng = np.random.default_rng(4)
    n, L = [4, 4, 4], [0, 12, 5]
    cache = Cache(rng, [4, 16, 9], 2, 8, 64, dtype).fill(rng, [4, 16, 9])
    path = np.array([bad, [0, 2, 3, -1], bad])
    want = [paged.compact(f64(x), cache.table, L, path, [0, 2, 0]) for x in (cache.k, cache.v)]
    status = zeros_status(3)
    lens = ttv.kv_compact_paged(cache.k, cache.v, cache.block_table, i32(L), i32([0, 4, 8, 12]), i32(path), i32([3, 2, 3]), status)
    assert status.tolist() == [-5, 0, -5] and lens.tolist() == [0, 15, 5]
    for x, y in zip((cache.k, cache.v), want):
        assert np.array_equal(f64(x), y, equal_nan=True)


def test_compaction_of_a_long_path_of_a_small_tree(gpu_lib):
    """128 entries that increase up to node 1 of two, at the end of the request's slots: their places lie behind the table."""
    rng = np.random.default_rng(4)
    cache = Cache(rng, [16], 2, 8, 64, F32).fill(rng, [16])
    path = [[0] + list(range(-125, 2))]
    before = [cache.k.clone(), cache.v.clone()]
    status = zeros_status(1)
    lens = ttv.kv_compact_paged(cache.k, cache.v, cache.block_table, i32([14]), i32([0, 2]), i32(path), i32([127]), status)
    assert status.tolist() == [-5] and lens.tolist() == [14]
    for x, y in zip((cache.k, cache.v), before):
        assert torch.equal(bits(x), bits(y))


def test_paths_of_more_requests_than_a_call_takes(gpu_lib):
    """65540 requests write and attend in one call each; their paths move in two, on slices of the arrays."""
    B, n, D = 65540, 3, 64
    rows, off, lens = torch.randn((B * n, 1, D), device="cuda"), i32(np.arange(B + 1) * n), i32(np.arange(B) % 5)
    kp, vp = (torch.zeros((B, 1, 8, D), device="cuda") for _ in range(2))
    table, status = i32(np.random.default_rng(0).permutation(B)[:, None]), zeros_status(B)
    ttv.rope_write_paged(None, rows, rows, kp, vp, table, lens, off, status)
    o = ttv.tree_attn_paged(rows, kp, vp, table, lens, off, None, 4, status, parents=i32(np.tile([-1, 0, 0], B)))
    assert o.isfinite().all()
    path, accept = i32(np.tile([0, 2], (B, 1))), i32(np.ones(B))
    want = [x[table[:, 0].long(), 0].clone() for x in (kp, vp)]
    at, row = lens.long(), torch.arange(B, device="cuda")
    for x in want:
        x[row, at + 1] = x[row, at + 2]
    with pytest.raises(ttv.SpecError, match="SHAPE"):
        ttv.kv_compact_paged(kp, vp, table, lens, off, path, accept, status)
    for b in (slice(0, 65535), slice(65535, B)):
        new = ttv.kv_compact_paged(kp, vp, table[b], lens[b], off[b.start:b.stop + 1], path[b], accept[b], status[b])
        assert torch.equal(new, lens[b] + 2)
    assert status.eq(0).all()
    for x, y in zip((kp, vp), want):
        assert torch.equal(x[table[:, 0].long(), 0], y)


# ------------------------------------------------------------------ together
def step(q, k, v, cache, rope, depth, parents, off, lens, path, accept, max_prefix, status, stream=None):
    """One step as a program runs it: rows into pages, attention, the accepted path."""
    table = cache.block_table if not hasattr(cache, "fixed") else cache.fixed
    turned = ttv.rope_write_paged(q, k, v, cache.k, cache.v, table, lens, off, status, rope, depth=depth, stream=stream)
    o = ttv.tree_attn_paged(turned, cache.k, cache.v, table, lens, off, None, max_prefix, status, parents=parents,
                            stream=stream)
    new = ttv.kv_compact_paged(cache.k, cache.v, table, lens, off, path, accept, status, stream=stream)
    return turned, o, new


@DTYPES
def test_steps_together(gpu_lib, dtype):
    """A prompt in two chunks, then two steps of trees, each against the oracle on the cache as it stands."""
    rng = np.random.default_rng(13)
    B, Hq, H, D, P = 2, 6, 2, 64, 16
    rope = ttv.rope_table(32, 10000.0, "yarn", 4.0, original=64.0)
    theta, scale = paged.frequencies(32, 10000.0, "yarn", 4.0, 64.0)
    cache = Cache(rng, [260, 200], H, P, D, dtype)
    kept = [f64(cache.k), f64(cache.v)]
    lens = [0, 0]
    status = zeros_status(B)
    for n, tree in (([70, 100], False), ([50, 0], False), ([12, 30], True), ([64, 9], True)):
        off = np.concatenate([[0], np.cumsum(n)])
        T = int(off[-1])
        q, k, v = (gpu(rng.standard_normal((T, h, D)), dtype) for h in (Hq, H, H))
        parents = [random_tree(rng, m) if m else [] for m in n] if tree else None
        flat = np.concatenate(parents).astype(int) if tree else None
        depth = np.concatenate([depths(p) for p in parents]).astype(int) if tree else None
        turned = ttv.rope_write_paged(q, k, v, cache.k, cache.v, cache.block_table, i32(lens), i32(off), status, rope,
                                      depth=i32(depth) if tree else None)
        assert_rotated(turned, q, paged.positions(lens, off, depth), theta, scale, False)
        keys = ttv.rope(k, rope, i32(lens), i32(off), status, depth=i32(depth) if tree else None)
        kept = [paged.write(kept[0], f64(keys), cache.table, lens, off), paged.write(kept[1], f64(v), cache.table, lens, off)]
        o = ttv.tree_attn_paged(turned, cache.k, cache.v, cache.block_table, i32(lens), i32(off), None, max(lens), status,
                                parents=i32(flat) if tree else None, causal=not tree)
        check_attn(o, turned, cache, lens, off, flat)
        if not tree:
            lens = [a + b for a, b in zip(lens, n)]
            continue
        paths = []
        for p in parents:
            node, path = len(p) - 1, []
            while node >= 0:
                path.append(node)
                node = p[node]
            paths.append(path[::-1])
        W = max(len(p) for p in paths)
        path, accept = np.array([p + [-1] * (W - len(p)) for p in paths]), [len(p) - 1 for p in paths]
        kept = [paged.compact(x, cache.table, lens, path, accept) for x in kept]
        lens = ttv.kv_compact_paged(cache.k, cache.v, cache.block_table, i32(lens), i32(off), i32(path), i32(accept),
                                    status).tolist()
        for x, y in zip((cache.k, cache.v), kept):
            assert np.array_equal(f64(x), y, equal_nan=True)
    assert status.eq(0).all()


def test_captured_and_on_two_streams(gpu_lib):
    """Two steps captured as graphs, the first calls of their kinds among them, replayed at once over changed inputs."""
    rng = np.random.default_rng(14)
    made = []
    for seed, (P, n) in enumerate(((16, 40), (64, 9))):
        r = np.random.default_rng(seed)
        Hq, H, D, L = 8, 4, 128, 500
        cache = Cache(r, [L + n], H, P, D, BF16).fill(r, [L])
        cache.fixed = cache.block_table
        tree = random_tree(r, n)
        path = [n - 1]
        while tree[path[0]] >= 0:
            path.insert(0, tree[path[0]])
        rows = [gpu(r.standard_normal((n, h, D)), BF16) for h in (Hq, H, H)]
        made.append(dict(cache=cache, rows=rows, tree=tree, n=n, L=L, args=(
            ttv.rope_table(D), i32(depths(tree)), i32(tree), i32([0, n]), i32([L]), i32([path]), i32([len(path) - 1]), L,
            zeros_status(1)), path=path))
    torch.cuda.synchronize()
    for m in made:
        m["graph"], m["stream"] = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(m["graph"], stream=m["stream"]):
            m["out"] = step(*m["rows"], m["cache"], *m["args"])
    for turn in range(3):
        before = []
        for m in made:
            for x in m["rows"]:
                x.copy_(torch.randn_like(x))
            before.append([f64(m["cache"].k), f64(m["cache"].v)])
        torch.cuda.synchronize()
        for m in made:
            with torch.cuda.stream(m["stream"]):
                m["graph"].replay()
        torch.cuda.synchronize()
        for m, old in zip(made, before):
            turned, o, new = m["out"]
            rope, depth, _, off, lens, _, accept, _, status = m["args"]
            assert status.item() == 0 and new.tolist() == [m["L"] + len(m["path"])]
            keys = ttv.rope(m["rows"][1], rope, lens, off, status, depth=depth)
            written = [paged.write(x, f64(y), m["cache"].table, [m["L"]], [0, m["n"]])
                       for x, y in zip(old, (keys, m["rows"][2]))]
            ref = paged.attn(f64(turned), *written, m["cache"].table, [m["L"]], [0, m["n"]], m["tree"])
            err = np.abs(f64(o) - ref[0])
            assert (err <= attn_bound(*ref, 128, BF16)).all()
            for x, y in zip((m["cache"].k, m["cache"].v), written):
                moved = paged.compact(y, m["cache"].table, [m["L"]], [m["path"]], [len(m["path"]) - 1])
                assert np.array_equal(f64(x), moved, equal_nan=True)


def test_calls_on_another_stream(gpu_lib):
    rng = np.random.default_rng(15)
    q, cache, off = batch(rng, [50], [400], 4, 2, 16, 128, BF16)
    status = zeros_status(1)
    args = (cache.k, cache.v, cache.block_table, i32([400]), i32(off), None, 400, status)
    want = ttv.tree_attn_paged(q, *args, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = ttv.tree_attn_paged(q, *args, causal=True, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)


def test_no_rows_at_all(gpu_lib):
    status = zeros_status(2)
    cache = Cache(np.random.default_rng(0), [16, 16], 2, 16, 64, BF16)
    none = i32([0, 0, 0])
    empty = lambda h: torch.empty((0, h, 64), dtype=BF16, device="cuda")  # noqa: E731
    assert ttv.rope(empty(2), ttv.rope_table(64), i32([0, 0]), none, status).shape == (0, 2, 64)
    assert ttv.rope_write_paged(empty(4), empty(2), empty(2), cache.k, cache.v, cache.block_table, i32([0, 0]), none,
                                status).shape == (0, 4, 64)
    assert ttv.tree_attn_paged(empty(4), cache.k, cache.v, cache.block_table, i32([0, 0]), none, None, 0, status,
                               causal=True).shape == (0, 4, 64)
    assert status.eq(0).all()


def test_first_calls_inside_a_capture(gpu_lib):
    """A fresh process whose first calls of every kind are captured, replayed twice."""
    code = """
import torch, token_tree_verification_gb300 as ttv
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
for dt, D in ((torch.bfloat16, 128), (torch.float32, 64)):
    kp, vp = (torch.zeros((20, 2, 16, D), dtype=dt, device="cuda") for _ in range(2))
    table = torch.arange(19, -1, -1, dtype=torch.int32, device="cuda").reshape(1, 20)
    rows = [torch.randn((150, h, D), device="cuda").to(dt) for h in (4, 2, 2)]
    off, lens, status, rope = i32(0, 150), i32(0), i32(0), ttv.rope_table(D)
    path, acc, at, tree = i32(0, 2).reshape(1, 2), i32(1), i32(10), i32(0, 64)
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        t = ttv.rope_write_paged(*rows, kp, vp, table, lens, off, status, rope)
        r = ttv.rope(rows[0], rope, lens, off, status)
        o = ttv.tree_attn_paged(t, kp, vp, table, lens, off, None, 0, status, causal=True)
        m = ttv.kv_compact_paged(kp, vp, table, at, tree, path, acc, status)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    kept = kp.clone()
    t2 = ttv.rope_write_paged(*rows, kp, vp, table, lens, off, status, rope)
    assert torch.equal(t, t2) and torch.equal(r, t2) and m.item() == 12
    assert torch.equal(o, ttv.tree_attn_paged(t2, kp, vp, table, lens, off, None, 0, status, causal=True))
    assert not torch.equal(kept, kp) and status.item() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]


@DTYPES
def test_pools_beyond_32_bits(gpu_lib, dtype):
    """Pages whose elements lie past 2^32 of the pool: written, attended to, moved."""
    rng = np.random.default_rng(16)
    H, P, D = 2, 4096, 128
    pages = 2 ** 32 // (H * P * D) + 3
    pools = [torch.empty((pages, H, P, D), dtype=dtype, device="cuda") for _ in range(2)]
    table = np.array([[pages - 1, 1], [2, pages - 2]])
    n, L = [20, 30], [4090, 4090]
    off = [0, 20, 50]
    q, k, v = (gpu(rng.standard_normal((50, h, D)), dtype) for h in (4, 2, 2))
    small = [torch.empty((4, H, P, D), dtype=dtype, device="cuda") for _ in range(2)]
    where = [pages - 1, 1, 2, pages - 2]
    for x, y in zip(pools, small):
        for i, page in enumerate(where):
            y[i] = gpu(rng.standard_normal((H, P, D)), dtype)
            x[page] = y[i]
    near = np.array([[0, 1], [2, 3]])
    path, acc = [[0, 3, 9]] * 2, [2, 2]
    got = []
    for kp, vp, t in ((*pools, table), (*small, near)):
        status = zeros_status(2)
        turned = ttv.rope_write_paged(q, k, v, kp, vp, i32(t), i32(L), i32(off), status, ttv.rope_table(D))
        o = ttv.tree_attn_paged(turned, kp, vp, i32(t), i32(L), i32(off), None, 4090, status, causal=True)
        lens = ttv.kv_compact_paged(kp, vp, i32(t), i32(L), i32(off), i32(path), i32(acc), status)
        assert status.eq(0).all() and lens.tolist() == [4093, 4093]
        got.append((turned, o))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for x, y in zip(pools, small):
        for i, page in enumerate(where):
            assert torch.equal(x[page], y[i])


def test_tensors_the_calls_refuse(gpu_lib):
    q, k, pool = (torch.zeros(s, dtype=BF16, device="cuda") for s in ((3, 4, 64), (3, 2, 64), (5, 2, 16, 64)))
    table, lens, off, st = i32([[0, 1]]), i32([0]), i32([0, 3]), zeros_status(1)
    rope = ttv.rope_table(64)
    attn = lambda q=q, kp=pool, vp=pool, t=table, lens=lens, off=off, st=st, **kw: ttv.tree_attn_paged(  # noqa: E731
        q, kp, vp, t, lens, off, None, 0, st, **({"causal": True} | kw))
    attn()
    for wrong in (dict(q=q.float()), dict(vp=pool.float()), dict(st=st.long()), dict(lens=lens.cpu()), dict(kp=pool.half(), vp=pool.half()),
                  dict(off=off.float())):
        with pytest.raises(TypeError):
            attn(**wrong)
    for wrong in (dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)), dict(t=table[0]), dict(t=i32([[0, 1], [2, 3]])), dict(kp=pool[0]),
                  dict(vp=pool[:4]), dict(causal=False), dict(parents=i32([0, 0, 0])), dict(o=q.float()), dict(off=i32([0])),
                  dict(t=table.long())):
        with pytest.raises(ValueError):
            attn(**wrong)
    with pytest.raises(ttv.SpecError):
        attn(kp=pool[:, :, :12].contiguous(), vp=pool[:, :, :12].contiguous())
    with pytest.raises(ValueError):
        ttv.rope(q, ttv.RopeTable(rope.freqs[:5], 1.0, 64), lens, off, st)
    with pytest.raises(TypeError):
        ttv.rope(q, rope, lens, off, st, out=q.float())
    with pytest.raises(ValueError):
        ttv.rope(q, rope, lens, off, st, depth=i32([0]))
    with pytest.raises(ttv.SpecError):
        ttv.rope(q, ttv.rope_table(128), lens, off, st)
    with pytest.raises(ttv.SpecError):                       # rows of the output on one another
        ttv.rope(q, rope, lens, off, st, out=torch.zeros((4, 64), dtype=BF16, device="cuda").expand(3, 4, 64))
    with pytest.raises(TypeError):
        ttv.rope_write_paged(q, k.float(), k, pool, pool.clone(), table, lens, off, st, rope)
    with pytest.raises(ValueError):
        ttv.rope_write_paged(q, k[:, :1], k, pool, pool.clone(), table, lens, off, st, rope)
    with pytest.raises(ValueError):
        ttv.rope_write_paged(None, k, k, pool, pool.clone(), table, lens, off, st, rope, q_out=q)
    with pytest.raises(ttv.SpecError):                       # the lengths may not be written where they are read
        ttv.kv_compact_paged(pool, pool.clone(), table, lens, off, i32([[0, 1]]), i32([1]), st, new_prefix_lens=lens)
    assert st.eq(0).all()
