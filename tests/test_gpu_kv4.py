"""The 4-bit KV cache on the GPU against its float64 oracle: writing and
reading are exact, attention is held to bounds counted in half steps of the
roundings it makes, and the calls run together as a step uses them."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import token_tree_verification_gb300 as ttv
from oracle import kv4

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def zeros_status(B):
    return torch.zeros(B, dtype=torch.int32, device="cuda")


def random_records(rng, shape, D):
    rec = rng.integers(0, 256, shape + (kv4.record_bytes(D),), dtype=np.uint8)
    rec[..., D:D + D // 8] = rng.integers(90, 110, shape + (D // 8,))
    return rec


def random_tree(rng, n, chain=False):
    return [-1] + [i - 1 if chain else int(rng.integers(max(0, i - 10), i)) for i in range(1, n)]


# ------------------------------------------------------------------ write, read
def crafted_rows(rng, T, H, D, dtype):
    """Rows of many sizes, with maxima and elements on and beside every kind of boundary."""
    x = rng.standard_normal((T, H, D)) * np.exp(3 * rng.standard_normal((T, H, 1)))
    g = x.reshape(-1, 16)
    n = g.shape[0]
    edge = np.concatenate([6 * (kv4.SCALES[:-1] + kv4.SCALES[1:]) / 2, [0, 61440, 1e30, 2.0 ** -130, 6e4]])
    pick = edge[rng.integers(0, len(edge), n)]
    near = np.float32(pick)
    sort = rng.integers(0, 4, n)
    near = np.where(sort == 1, np.nextafter(near, np.float32(np.inf)), np.where(sort == 2, np.nextafter(near, np.float32(0)), near))
    use = sort < 3
    g[use] = np.clip(g[use], -1, 1) * np.abs(near[use, None])
    g[use, 3] = near[use]
    # elements on the boundaries between codes of their group's scale
    _, byte, _ = kv4.quantise(x.astype(np.float32).reshape(-1, 16))
    s = kv4.SCALES[byte[:, 0]]
    for j, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        e = np.float32(s * mid)
        e = np.where(sort == 1, np.nextafter(e, np.float32(np.inf)), np.where(sort == 2, np.nextafter(e, np.float32(0)), e))
        g[:, 5 + j] = np.where(rng.random(n) < 0.7, e * rng.choice([-1, 1], n), g[:, 5 + j])
    g[rng.random(n) < 0.05] = 0.0
    return torch.from_numpy(np.clip(x, -3e38, 3e38).astype(np.float32)).to(dtype)


@DTYPES
@pytest.mark.parametrize("D,H,counts,start,cap", [
    (128, 3, [5, 1, 9], [0, 7, 30], 40), (64, 1, [3, 0, 6], [2, 0, 9], 15), (64, 5, [17], [3], 33),
    (128, 8, [70, 200, 1, 0, 33], [0, 5, 399, 400, 1], 400), (128, 1, [1], [0], 1)])
def test_write_and_read_are_exact(dtype, D, H, counts, start, cap):
    rng = np.random.default_rng(len(counts) * 131 + D)
    off = np.concatenate([[0], np.cumsum(counts)])
    T, B = int(off[-1]), len(counts)
    k, v = crafted_rows(rng, T + 2, H, D, dtype), crafted_rows(rng, T + 2, H, D, dtype)   # two rows behind the last request
    before = rng.integers(0, 256, (B, H, cap, kv4.record_bytes(D)), dtype=np.uint8)
    cache, st = torch.from_numpy(before.copy()).cuda(), zeros_status(B)
    ttv.kv4_write(k.cuda(), v.cuda(), cache, i32(start), i32(off), st)
    want = before.copy()
    kv4.write(want, k.float().numpy(), v.float().numpy(), start, off)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    assert st.tolist() == [0] * B
    kw, vw = kv4.read(want, D, start, off)
    for out_type in (BF16, F32):
        rows = [torch.full((T + 2, H, D), -7.0, dtype=out_type, device="cuda") for _ in range(2)]
        ttv.kv4_read(cache, i32(start), i32(off), st, out=rows)
        for got, ref in zip(rows, (kw, vw)):
            np.testing.assert_array_equal(got[:T].double().cpu().numpy(), ref)
            assert (got[T:] == -7.0).all()
    assert st.tolist() == [0] * B


@DTYPES
def test_rows_inside_other_tensors(dtype):
    """Rows of a fused projection in, and slots out into a dense [B][Hkv][S][D] cache."""
    rng = np.random.default_rng(3)
    T, H, D, cap = 37, 4, 128, 50
    fused = torch.from_numpy(rng.standard_normal((T, 3 * H, D)).astype(np.float32)).to(dtype).cuda()
    k, v = fused[:, H:2 * H], fused[:, 2 * H:]
    heads_first = v.transpose(0, 1).contiguous().transpose(0, 1)     # another order of strides
    cache, st = ttv.make_kv4_cache(1, H, cap, D), zeros_status(1)
    ttv.kv4_write(k, heads_first, cache, i32([4]), i32([0, T]), st)
    want = np.zeros(cache.shape, np.uint8)
    kv4.write(want, k.float().cpu().numpy(), v.float().cpu().numpy(), [4], [0, T])
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    dense = torch.full((2, 1, H, cap, D), 5.0, dtype=dtype, device="cuda")
    out = (dense[0, 0].transpose(0, 1)[4:4 + T], dense[1, 0].transpose(0, 1)[4:4 + T])
    ttv.kv4_read(cache, i32([4]), i32([0, T]), st, out=out)
    ref = kv4.values(want[0, :, 4:4 + T], D)
    for got, r in zip(dense[:, 0], ref):
        np.testing.assert_array_equal(got[:, 4:4 + T].double().cpu().numpy(), r)
        assert (got[:, :4] == 5).all() and (got[:, 4 + T:] == 5).all()
    # a row that every token shares
    ttv.kv4_write(k[:1].expand(T, H, D), v, cache, i32([4]), i32([0, T]), st)
    kv4.write(want, k[:1].expand(T, H, D).float().cpu().numpy(), v.float().cpu().numpy(), [4], [0, T])
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    assert st.tolist() == [0]


@DTYPES
def test_rows_with_nan_or_infinity_are_reported(dtype):
    rng = np.random.default_rng(4)
    off, start, H, D = [0, 6, 12, 20], [0, 3, 1], 2, 64
    k, v = (torch.from_numpy(rng.standard_normal((20, H, D)).astype(np.float32)).to(dtype) for _ in range(2))
    k[2, 1, 17], v[13, 0, 0], v[14, 1, 63] = float("nan"), float("inf"), float("-inf")
    cache, st = ttv.make_kv4_cache(3, H, 16, D), zeros_status(3)
    ttv.kv4_write(k.cuda(), v.cuda(), cache, i32(start), i32(off), st)
    assert st.tolist() == [-13, 0, -13]
    want = np.zeros(cache.shape, np.uint8)
    for x in (k, v):       # the groups that hold one become zeros
        g = x.view(20, H, D // 16, 16)
        g[~torch.isfinite(g).all(-1)] = 0
    kv4.write(want, k.float().numpy(), v.float().numpy(), start, off)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("off,start,codes", [
    ([0, 4, 8], [0, 13], [0, -10]), ([0, 4, 8], [-1, 0], [-10, 0]), ([0, 5, 3], [0, 0], [0, -4]),
    ([-1, 4, 8], [0, 0], [-4, 0]), ([0, 4, 9], [0, 0], [0, -4]), ([0, 4, 8], [2 ** 31 - 1, 0], [-10, 0])])
def test_a_request_in_error_changes_nothing(off, start, codes):
    rng = np.random.default_rng(5)
    H, D, cap = 2, 64, 16
    k = torch.from_numpy(rng.standard_normal((8, H, D)).astype(np.float32)).cuda()
    before = rng.integers(0, 256, (2, H, cap, kv4.record_bytes(D)), dtype=np.uint8)
    cache, st = torch.from_numpy(before).cuda(), zeros_status(2)
    ttv.kv4_write(k, k, cache, i32(start), i32(off), st)
    assert st.tolist() == codes
    after = cache.cpu().numpy()
    for b in range(2):
        if codes[b]:
            np.testing.assert_array_equal(after[b], before[b])
    rows = torch.full((2, 8, H, D), 3.0, device="cuda")
    st2 = zeros_status(2)
    ttv.kv4_read(cache, i32(start), i32(off), st2, out=(rows[0], rows[1]))
    assert st2.tolist() == codes
    good = [b for b in range(2) if not codes[b]]
    touched = {t for b in good for t in range(off[b], off[b + 1])}
    for t in set(range(8)) - touched:
        assert (rows[:, t] == 3.0).all(), t


# ------------------------------------------------------------------ attention
def check_attn(q, rec, L, off, parents, window=0, sinks=0, masks="mask", scale=0.0, max_prefix=None,
               stored=None):
    """`stored`: what the cache holds where that is not what the rows see of it, `rec`."""
    dtype, D = q.dtype, q.shape[2]
    st = zeros_status(len(L))
    args = (q.cuda(), torch.from_numpy(rec if stored is None else stored).cuda(), i32(L), i32(off))
    par = i32(parents)
    mask = ttv.build_tree_mask(par, i32(off), st)[0] if masks == "mask" else None
    o = ttv.tree_attn_kv4(*args, mask, int(max(L)) if max_prefix is None else max_prefix, st, softmax_scale=scale,
                          parents=None if mask is not None else par, window=window, sinks=sinks)
    got = o.double().cpu().numpy()
    assert st.tolist() == [0] * len(L)
    ref, size, big, reach = kv4.tree_attn(q.float().numpy(), rec, L, off, parents, window, sinks, scale or None)
    # Scores: every product is exact (bf16) or off by 2^-22 (two halves of an fp32 query), sums of D
    # products in fp32 lose at most D 2^-24 of sum |q||k|, and the exponential 2^-20: a weight is off by the
    # factor 1 + delta, and its normaliser by as much.
    delta = (2.0 ** -21 + D * 2.0 ** -24) * big[..., None] + 2.0 ** -20
    # Weights: one half (half a step, 2^-11) or two (2^-22); sums over the keys in fp32, 2^-18 of the total.
    weight = 2.0 ** -11 if dtype == BF16 else 2.0 ** -22
    last = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24      # half a step of the output
    # A half's smallest step is 2^-24.  Weights are scaled so that a row's largest is 2^7 or more, so each is
    # off by at most 2^-25 / 2^7 = 2^-32 of the largest (a smaller one may be lost whole), and the largest is
    # at most the normaliser.
    tol = size * (2 * delta + weight + 2.0 ** -18) + last * np.abs(ref) * 1.01 + 2.0 ** -32 * reach
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], (np.abs(got - ref) / tol)[bad].max())
    return o


SHAPES = [  # D, Hq, Hkv, prefixes, nodes
    (128, 1, 1, [0], [1]), (64, 1, 1, [1], [1]), (128, 4, 4, [15, 16, 17], [1, 1, 1]), (64, 8, 1, [63, 64, 65, 0], [2, 1, 3, 5]),
    (128, 8, 1, [300], [1]), (128, 3, 1, [129, 5], [7, 40]), (128, 10, 2, [33], [13]), (64, 4, 2, [700, 20, 0], [64, 33, 16]),
    (128, 2, 2, [1000], [128]), (128, 16, 2, [250, 511], [128, 3]), (64, 32, 1, [90], [11]), (128, 128, 1, [70], [3]),
    (128, 5, 1, [4000], [26]), (128, 32, 32, [2048], [9]), (64, 2, 1, [20000], [2]),
    # 48 and 64 rows on a key
    (128, 4, 1, [600], [12]), (64, 16, 2, [10, 300], [8, 8]), (128, 2, 2, [1500], [64]),
    # splits into 16, for one row block
    (128, 1, 1, [9000], [20]), (64, 2, 2, [9000], [90])]

RAGGED = [  # one request with many more rows than the mean, which its CTAs take in turns
    (128, 2, 2, [3000, 10, 5, 2000], [1, 1, 1, 20]), (128, 1, 1, [1900, 2000], [1, 60]),
    (64, 2, 1, [3000, 3, 0], [128, 1, 1]), (128, 8, 2, [40, 2, 300, 1, 0], [1, 1, 128, 1, 1]),
    (64, 1, 1, [0, 0, 0, 1500], [1, 1, 1, 100])]


@DTYPES
@pytest.mark.parametrize("D,Hq,Hkv,L,n", SHAPES + RAGGED)
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3), (1, 0)], ids=["all", "window", "self"])
def test_attention(dtype, D, Hq, Hkv, L, n, window, sinks):
    rng = np.random.default_rng(Hq * 7 + L[0] + n[0])
    off = np.concatenate([[0], np.cumsum(n)])
    S = max(a + b for a, b in zip(L, n)) + 3
    rec = random_records(rng, (len(L), Hkv, S), D)
    for b, (a, c) in enumerate(zip(L, n)):
        rec[b, :, a + c:] = 255             # slots nobody wrote: NaN, were they decoded
    parents = sum((random_tree(rng, c) for c in n), [])
    q = torch.from_numpy((2 * rng.standard_normal((off[-1], Hq, D))).astype(np.float32)).to(dtype)
    a = check_attn(q, rec, L, off, parents, window, sinks, "mask")
    b = check_attn(q, rec, L, off, parents, window, sinks, "parents", max_prefix=max(L) + 1000)
    if dtype == F32:
        np.testing.assert_allclose(a.cpu().numpy(), b.cpu().numpy(), rtol=1e-3, atol=1e-4)


@DTYPES
@pytest.mark.parametrize("window,sinks", [(2, 0), (5, 40), (200, 70), (64, 64), (10 ** 9, 10 ** 9), (33, 129)])
@pytest.mark.parametrize("chain", [False, True])
def test_windows_that_cut_the_tree_and_the_tiles(dtype, window, sinks, chain):
    rng = np.random.default_rng(window + sinks)
    L, n, D = [130, 0, 40, 300], [100, 128, 5, 1], 64
    off = np.concatenate([[0], np.cumsum(n)])
    rec = random_records(rng, (4, 2, 305), D)
    parents = sum((random_tree(rng, c, chain) for c in n), [])
    q = torch.from_numpy(rng.standard_normal((off[-1], 6, D)).astype(np.float32)).to(dtype)
    check_attn(q, rec, L, off, parents, window, sinks)


@DTYPES
@pytest.mark.parametrize("Hq,n", [(2, [1, 3, 2]), (4, [6, 8, 1]), (4, [16, 13, 1]), (8, [40, 5, 22])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (30, 5), (129, 64)])
def test_slots_behind_the_window_may_hold_anything(dtype, Hq, n, window, sinks):
    rng = np.random.default_rng(Hq + window)
    L, D = [500, 70, 263], 128
    off = np.concatenate([[0], np.cumsum(n)])
    rec = random_records(rng, (3, 1, 560), D)
    stored = rec.copy()
    for b, (a, c) in enumerate(zip(L, n)):
        stored[b, :, sinks:max(sinks, a - window + 1)] = 255      # the root's window begins at a - window + 1
        stored[b, :, a + c:] = 255
    parents = sum((random_tree(rng, c) for c in n), [])
    q = torch.from_numpy(rng.standard_normal((off[-1], Hq, D)).astype(np.float32)).to(dtype)
    check_attn(q, rec, L, off, parents, window, sinks, stored=stored)


@DTYPES
def test_large_scores_and_far_values(dtype):
    """Score ranges that move the softmax's reference, and queries and values at the ends of their range."""
    rng = np.random.default_rng(11)
    L, n, D = [500, 200], [6, 20], 128
    off = np.concatenate([[0], np.cumsum(n)])
    rec = random_records(rng, (2, 2, 520), D)
    rec[0, :, 100:400:7, D:D + 8] = 130                    # some keys 16 times as large
    rec[1, :, :, D + 8:D + 16] = rng.integers(0, 227, rec[1, :, :, D + 8:D + 16].shape)   # values of every size
    parents = sum((random_tree(rng, c) for c in n), [])
    q = rng.standard_normal((off[-1], 4, D))
    q[3] *= 30
    q[7] *= 1e-6
    q[9] *= 1e5
    q[9, :, ::2] *= 1e-9
    q[11] = 0
    q = torch.from_numpy(q.astype(np.float32)).to(dtype)
    check_attn(q, rec, L, off, parents, scale=0.05)
    check_attn(q[:6], rec[:1], L[:1], off[:2], parents[:6], scale=0.2)


@DTYPES
def test_rows_that_see_nothing_and_rows_with_nan(dtype):
    rng = np.random.default_rng(12)
    D, n = 128, 20
    rec = torch.from_numpy(random_records(rng, (1, 1, 40), D)).cuda()
    q = torch.from_numpy(rng.standard_normal((n, 4, D)).astype(np.float32)).to(dtype).cuda()
    off, st = i32([0, n]), zeros_status(1)
    par = i32(random_tree(rng, n))
    mask, _ = ttv.build_tree_mask(par, off, st)
    ref = ttv.tree_attn_kv4(q, rec, i32([0]), off, mask, 0, st)
    mask[5] = 0
    q[9, 2, 77] = float("nan")
    got = ttv.tree_attn_kv4(q, rec, i32([0]), off, mask, 0, st)
    assert (got[5] == 0).all() and torch.isnan(got[9, 2]).all()
    ref[5], ref[9, 2], got[9, 2] = 0, 0, 0
    assert torch.equal(got, ref)
    assert st.tolist() == [0]


@DTYPES
def test_attention_reports_and_leaves_a_request_in_error(dtype):
    rng = np.random.default_rng(13)
    D = 64
    rec = torch.from_numpy(random_records(rng, (3, 2, 50), D)).cuda()
    q = torch.from_numpy(rng.standard_normal((24, 4, D)).astype(np.float32)).to(dtype).cuda()
    parents = random_tree(rng, 8) + random_tree(rng, 8) + random_tree(rng, 8)
    good = ttv.tree_attn_kv4(q, rec, i32([20, 30, 5]), i32([0, 8, 16, 24]), None, 40, zeros_status(3), parents=i32(parents))
    for L, off, codes in (([20, 43, 5], [0, 8, 16, 24], [0, -10, 0]), ([20, -1, 5], [0, 8, 16, 24], [0, -10, 0]),
                          ([20, 30, 5], [0, 8, 8, 24], [0, -4, 0])):
        st = zeros_status(3)
        o = torch.full_like(q, 9.0)
        ttv.tree_attn_kv4(q, rec, i32(L), i32(off), None, 40, st, o=o, parents=i32(parents))
        assert st.tolist()[:2] == codes[:2]
        assert torch.equal(o[:8], good[:8])
        if codes[1] == -10:
            assert (o[8:16] == 9.0).all() and torch.equal(o[16:], good[16:]) and st.tolist() == codes
    st = zeros_status(3)
    ttv.tree_attn_kv4(q, rec, i32([20, 2 ** 31 - 1, 5]), i32([0, 8, 16, 24]), None, 40, st, parents=i32(parents))
    assert st.tolist() == [0, -10, 0]
    bad = list(parents)
    bad[10] = 5
    st = zeros_status(3)
    o = ttv.tree_attn_kv4(q, rec, i32([20, 30, 5]), i32([0, 8, 16, 24]), None, 40, st, parents=i32(bad))
    assert st.tolist() == [0, -5, 0] and torch.equal(o[:8], good[:8]) and torch.equal(o[16:], good[16:])


@DTYPES
def test_many_requests_and_empty_ones(dtype):
    """300 requests of 0 to 3 rows: offsets longer than a block, looked up from any row."""
    rng = np.random.default_rng(20)
    B, H, D, cap = 300, 2, 64, 12
    n = rng.integers(0, 4, B)
    n[:2], n[-1] = 0, 0
    off, start = np.concatenate([[0], np.cumsum(n)]), rng.integers(0, 9, B)
    T = int(off[-1])
    k, v = (torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(dtype) for _ in range(2))
    cache, st = ttv.make_kv4_cache(B, H, cap, D), zeros_status(B)
    ttv.kv4_write(k.cuda(), v.cuda(), cache, i32(start), i32(off), st)
    want = np.zeros(cache.shape, np.uint8)
    kv4.write(want, k.float().numpy(), v.float().numpy(), start, off)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    kk, _ = ttv.kv4_read(cache, i32(start), i32(off), st, rows=T, dtype=dtype)
    np.testing.assert_array_equal(kk.double().cpu().numpy(), kv4.read(want, D, start, off)[0])
    # no rows at all: nothing is launched
    none = torch.empty((0, H, D), dtype=dtype, device="cuda")
    ttv.kv4_write(none, none, cache, i32(start), torch.zeros(B + 1, dtype=torch.int32, device="cuda"), st)
    assert ttv.kv4_read(cache, i32(start), torch.zeros(B + 1, dtype=torch.int32, device="cuda"), st, rows=0)[0].shape[0] == 0
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    assert not st.any()


def test_long_runs_of_rows():
    """Enough rows that a warp walks several turns of them, over tokens, heads and requests."""
    rng = np.random.default_rng(21)
    for D, H, n in ((128, 3, [9000, 0, 4321]), (64, 32, [1, 2500])):
        off = np.concatenate([[0], np.cumsum(n)])
        T, start = int(off[-1]), [3] * len(n)
        k, v = (torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(BF16) for _ in range(2))
        cache, st = ttv.make_kv4_cache(len(n), H, max(n) + 4, D), zeros_status(len(n))
        ttv.kv4_write(k.cuda(), v.cuda(), cache, i32(start), i32(off), st)
        want = np.zeros(cache.shape, np.uint8)
        kv4.write(want, k.float().numpy(), v.float().numpy(), start, off)
        np.testing.assert_array_equal(cache.cpu().numpy(), want)
        kk, vv = ttv.kv4_read(cache, i32(start), i32(off), st, rows=T, dtype=F32)
        for got, ref in zip((kk, vv), kv4.read(want, D, start, off)):
            np.testing.assert_array_equal(got.double().cpu().numpy(), ref)
        assert not st.any()


def test_two_streams_at_once():
    """Calls on two streams, each with its own outputs, while the other runs."""
    rng = np.random.default_rng(22)
    L, n, D = [900, 2000], [1, 40], 128
    cache = torch.from_numpy(random_records(rng, (2, 4, 2050), D)).cuda()
    q = [torch.from_numpy(rng.standard_normal((c, 8, D)).astype(np.float32)).to(BF16).cuda() for c in (2, 80, 256)]
    batches = []
    for x in q:
        c = x.shape[0] // 2
        par = random_tree(rng, c) + random_tree(rng, c)
        batches.append((x, i32(L), i32([0, c, 2 * c]), i32(par), zeros_status(2)))
    cache = torch.cat([cache, cache], 2)[:, :, :2200].contiguous()
    call = lambda x, lens, off, par, st: ttv.tree_attn_kv4(x, cache, lens, off, None, 2000, st, parents=par)  # noqa: E731
    ref = [call(*b) for b in batches]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(24):
        with torch.cuda.stream(streams[i % 2]):
            got.append((i % 3, call(*batches[i % 3])))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref[j]) for j, o in got)
    assert not any(b[4].any() for b in batches)


@pytest.mark.parametrize("G", [1, 12, 24, 40])
def test_as_many_requests_and_heads_as_a_launch_takes(G):
    """65535 (request, head) pairs, a tile of keys each, against calls for a few of the requests."""
    rng = np.random.default_rng(24)
    B, H, D, cap = 257, 255, 64, 6
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randint(0, 256, (B, H, cap, 80), dtype=torch.uint8, device="cuda", generator=gen)
    cache[..., D:D + D // 8] = torch.randint(92, 107, (B, H, cap, D // 8), dtype=torch.uint8, device="cuda", generator=gen)
    q = torch.randn((B, H * G, D), device="cuda", generator=gen).to(BF16)
    L, off, par, st = i32(rng.integers(0, cap, B)), i32(np.arange(B + 1)), i32([-1] * B), zeros_status(B)
    o = ttv.tree_attn_kv4(q, cache, L, off, None, cap, st, parents=par)
    for b in (0, 128, 254):
        few = ttv.tree_attn_kv4(q[b:b + 3], cache[b:b + 3], L[b:b + 3], off[:4], None, cap, st[:3], parents=par[:3])
        assert torch.equal(o[b:b + 3], few)
    assert not st.any()


def test_outputs_made_for_a_call_on_another_stream():
    """An output dropped while its call is under way on another stream is not handed out again before."""
    rng = np.random.default_rng(23)
    cache, n = torch.from_numpy(random_records(rng, (1, 8, 9000), 128)).cuda(), 9000
    start, off, st = i32([0]), i32([0, n]), zeros_status(1)
    side = torch.cuda.Stream()
    ref = ttv.kv4_read(cache, start, off, st, rows=n)
    q = torch.from_numpy(rng.standard_normal((1, 8, 128)).astype(np.float32)).to(BF16).cuda()
    want = ttv.tree_attn_kv4(q, cache, i32([n - 1]), i32([0, 1]), None, n, st, parents=i32([-1]))
    lens, one, par = i32([n - 1]), i32([0, 1]), i32([-1])
    torch.cuda.synchronize()
    for _ in range(5):
        for _ in range(3):
            k, v = ttv.kv4_read(cache, start, off, st, rows=n, stream=side)
            o = ttv.tree_attn_kv4(q, cache, lens, one, None, n, st, parents=par, stream=side)
            addresses = {k.data_ptr(), v.data_ptr(), o.data_ptr()}
            del k, v, o
            fresh = [torch.empty_like(ref[0]), torch.empty_like(ref[1]), torch.empty_like(want)]
            busy = not side.query()
            assert not (busy and addresses & {x.data_ptr() for x in fresh})
        side.synchronize()
    k, v = ttv.kv4_read(cache, start, off, st, rows=n, stream=side)
    o = ttv.tree_attn_kv4(q, cache, lens, one, None, n, st, parents=par, stream=side)
    side.synchronize()
    assert torch.equal(k, ref[0]) and torch.equal(v, ref[1]) and torch.equal(o, want) and st.tolist() == [0]


def test_as_many_rows_as_can_be_counted():
    """2^31 - 1 rows (one, broadcast), all but three of them behind the last request."""
    rng = np.random.default_rng(22)
    T, D, cap = 2 ** 31 - 1, 64, 8
    k = torch.from_numpy(rng.standard_normal((1, 1, D)).astype(np.float32)).to(BF16)
    before = rng.integers(0, 256, (2, 1, cap, kv4.record_bytes(D)), dtype=np.uint8)
    cache, st = torch.from_numpy(before).cuda(), zeros_status(2)
    wide = k.cuda().expand(T, 1, D)
    ttv.kv4_write(wide, wide, cache, i32([4, 1]), i32([0, 2, 3]), st)
    three = k.float().expand(3, 1, D).numpy()
    kv4.write(before, three, three, [4, 1], [0, 2, 3])
    np.testing.assert_array_equal(cache.cpu().numpy(), before)
    assert st.tolist() == [0, 0]


def test_cache_offsets_beyond_32_bits():
    """The second head of a cache of 4.8 GB: slots near its end, by window."""
    D, cap = 128, 1 << 24
    cache = torch.zeros((1, 2, cap, 144), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(14)
    L, n = cap - 300, 12
    k, v = (torch.from_numpy(rng.standard_normal((200 + n, 2, D)).astype(np.float32)).cuda() for _ in range(2))
    st = zeros_status(1)
    ttv.kv4_write(k, v, cache, i32([L - 200]), i32([0, 200 + n]), st)
    kk, vv = ttv.kv4_read(cache, i32([L - 200]), i32([0, 200 + n]), st, rows=200 + n, dtype=F32)
    small = np.zeros((1, 2, 200 + n, 144), np.uint8)
    kv4.write(small, k.cpu().numpy(), v.cpu().numpy(), [0], [0, 200 + n])
    np.testing.assert_array_equal(kk.double().cpu().numpy(), kv4.read(small, D, [0], [0, 200 + n])[0])
    parents = random_tree(rng, n)
    for dtype in (BF16, F32):
        for Hq in (4, 40):
            q = torch.from_numpy(rng.standard_normal((n, Hq, D)).astype(np.float32)).to(dtype)
            o = ttv.tree_attn_kv4(q.cuda(), cache, i32([L]), i32([0, n]), None, L, st, parents=i32(parents), window=150)
            ref, size, _, _ = kv4.tree_attn(q.float().numpy(), small, [200], [0, n], parents, window=150)
            assert (np.abs(o.double().cpu().numpy() - ref) <= 2.0 ** -7 * size).all()
    newp = ttv.kv4_compact(cache, i32([L]), i32([0, n]), i32([[0, 3, 7]]), i32([2]), st)
    assert newp.tolist() == [L + 3] and st.tolist() == [0]
    np.testing.assert_array_equal(cache[0, :, L + 1:L + 3].cpu().numpy(), small[0][:, [203, 207]])
    del cache


# ------------------------------------------------------------------ compaction, the step
def test_compact_moves_records_as_the_oracle_moves_rows():
    rng = np.random.default_rng(15)
    for D in (64, 128):
        off, L, W = np.array([0, 9, 30, 31, 60], np.int32), np.array([3, 40, 0, 17], np.int32), 8
        rec = rng.integers(0, 256, (4, 3, 80, kv4.record_bytes(D)), dtype=np.uint8)
        path = np.full((4, W), -1, np.int32)
        path[0, :3], path[1], path[2, :1], path[3, :4] = [0, 2, 3], [0, 1, 5, 6, 9, 12, 18, 20], [0], [0, 4, 10, 28]
        acc = np.array([2, 7, 0, 3], np.int32)
        for pre in ([0, 0, 0, 0], [0, -9, 0, 0]):
            want, newp, sto = oracle.kv_compact(rec.view(np.float32), L, off, path, acc, np.array(pre, np.int32))
            cache, st = torch.from_numpy(rec).cuda(), i32(pre)
            got = ttv.kv4_compact(cache, i32(L), i32(off), i32(path), i32(acc), st)
            np.testing.assert_array_equal(got.cpu().numpy(), newp)
            np.testing.assert_array_equal(st.cpu().numpy(), sto)
            np.testing.assert_array_equal(cache.cpu().numpy().view(np.float32).view(np.uint8), np.asarray(want).view(np.uint8))
    # malformed paths, and a tree that does not fit
    path = i32([[0, 3, 3, -1], [1, 2, -1, -1], [0, 1, -1, -1], [0, 1, 2, -1]])
    st, cache = zeros_status(4), torch.from_numpy(rec[:, :, :40].copy()).cuda()
    before = cache.clone()
    newp = ttv.kv4_compact(cache, i32([2, 2, 36, 2]), i32([0, 6, 12, 18, 24]), path, i32([2, 1, 1, 9]), st)
    assert st.tolist() == [-5, -5, -10, -4] and newp.tolist() == [2, 2, 36, 2] and torch.equal(cache, before)
    # a prefix whose sum with the tree passes 2^31
    st = zeros_status(4)
    ttv.kv4_compact(cache, i32([2, 2 ** 31 - 1, 2 ** 31 - 6, 2]), i32([0, 6, 12, 18, 24]), i32([[0, 1, -1, -1]] * 4), i32([1] * 4), st)
    assert st.tolist() == [0, -10, -10, 0] and torch.equal(cache, before)


def step_inputs(seed, B, Hq, Hkv, D, n, V, steps):
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    return [dict(q=f(B * n, Hq, D), k=f(B * n, Hkv, D), v=f(B * n, Hkv, D), target=3 * f(B * n, V),
                 parents=np.concatenate([random_tree(rng, n) for _ in range(B)]),
                 tokens=rng.integers(0, V, B * n)) for _ in range(steps)]


@DTYPES
def test_decoding_steps_run_together(dtype):
    """Prompts written, then steps of tree write, attention, verification and compaction, against the same
    steps on the oracle's cache; eager and replayed as a captured graph on another stream."""
    B, Hq, Hkv, D, n, V, cap = 3, 8, 2, 128, 12, 40, 120
    rng = np.random.default_rng(16)
    prompt = [30, 0, 47]
    poff = np.concatenate([[0], np.cumsum(prompt)])
    pk, pv = (torch.from_numpy(rng.standard_normal((poff[-1], Hkv, D)).astype(np.float32)).to(dtype) for _ in range(2))
    steps = step_inputs(17, B, Hq, Hkv, D, n, V, 4)
    for s in steps:                    # tokens that the target often picks, so that paths are accepted
        best = s["target"].argmax(-1)
        for b in range(B):
            for i in range(1, n):
                if rng.random() < 0.7:
                    s["tokens"][b * n + i] = best[b * n + s["parents"][b * n + i]]
    off = np.arange(B + 1) * n
    W = n + 1

    cuda = lambda x, t=dtype: torch.as_tensor(x).to(t).cuda()  # noqa: E731

    def on_gpu(graph):
        cache, st = ttv.make_kv4_cache(B, Hkv, cap, D), zeros_status(B)
        lens, ws = i32(prompt), ttv.make_verify_workspace(B, B * n, V)
        ttv.kv4_write(pk.cuda(), pv.cuda(), cache, i32([0] * B), i32(poff), st)
        buf = {x: cuda(steps[0][x], torch.int32 if x in ("parents", "tokens") else torch.float32 if x == "target" else dtype)
               for x in steps[0]}
        doff, new, o = i32(off), torch.empty_like(lens), torch.empty_like(buf["q"])

        def one():
            mask, _ = ttv.build_tree_mask(buf["parents"], doff, st)
            ttv.kv4_write(buf["k"], buf["v"], cache, lens, doff, st)
            ttv.tree_attn_kv4(buf["q"], cache, lens, doff, mask, cap - n, st, o=o, window=40, sinks=2)
            r = ttv.tree_verify(buf["target"], None, buf["tokens"], buf["parents"], doff, 0.0, 1, W, st, ws)
            ttv.kv4_compact(cache, lens, doff, r["path_nodes"], r["accept_len"], st, new_prefix_lens=new)
            lens.copy_(new)
            return r

        got, g, side = [], None, torch.cuda.Stream()
        for i, s in enumerate(steps):
            for x in s:
                buf[x].copy_(cuda(s[x], buf[x].dtype))
            torch.cuda.synchronize()
            if graph and i == 1:
                g = torch.cuda.CUDAGraph()
                keep = (cache.clone(), lens.clone())
                with torch.cuda.graph(g):
                    r = one()
                torch.cuda.synchronize()
                assert torch.equal(cache, keep[0]) and torch.equal(lens, keep[1])
            with torch.cuda.stream(side if graph else torch.cuda.current_stream()):
                if g is None:
                    r = one()
                else:
                    g.replay()
            torch.cuda.synchronize()
            got.append((o.clone(), r["accept_len"].clone(), lens.clone()))
        assert st.tolist() == [0] * B
        return got, cache.cpu().numpy()

    eager, cache = on_gpu(False)
    replayed, cache2 = on_gpu(True)
    np.testing.assert_array_equal(cache, cache2)
    for a, b in zip(eager, replayed):
        assert all(torch.equal(x, y) for x, y in zip(a, b))

    ref, L = np.zeros_like(cache), np.array(prompt)
    kv4.write(ref, pk.float().numpy(), pv.float().numpy(), [0] * B, poff)
    for s, (o, acc, lens) in zip(steps, eager):
        rounded = {x: torch.from_numpy(s[x]).to(dtype).float().numpy() for x in ("q", "k", "v")}
        kv4.write(ref, rounded["k"], rounded["v"], L, off)
        want, size, _, _ = kv4.tree_attn(rounded["q"], ref, L, off, s["parents"], 40, 2)
        assert (np.abs(o.double().cpu().numpy() - want) <= (2.0 ** -7 if dtype == BF16 else 2.0 ** -14) * size).all()
        w = oracle.tree_verify(s["target"], None, s["tokens"].astype(np.int32), s["parents"].astype(np.int32),
                               off.astype(np.int32), 0.0, 1, W)
        np.testing.assert_array_equal(acc.cpu().numpy(), w["accept_len"])
        for b in range(B):
            a = int(w["accept_len"][b])
            src = [L[b] + x for x in w["path_nodes"][b, 1:a + 1]]
            ref[b, :, L[b] + 1:L[b] + 1 + a] = ref[b][:, src].copy()
        L = L + 1 + w["accept_len"]
        np.testing.assert_array_equal(lens.cpu().numpy(), L)
    assert sum(int(a.sum()) for _, a, _ in eager) > 0
    np.testing.assert_array_equal(cache, ref)


FIRST_CALLS = """
import torch, token_tree_verification_gb300 as ttv
torch.manual_seed(0)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
L, cap = 3000, 3200
cache = ttv.make_kv4_cache(1, 2, cap, 128)
k, v = torch.randn(2, L + 128, 2, 128, device="cuda").bfloat16()
zero, st = i32([0]), i32([0])
runs = [(torch.randn(n, 2 * g, 128, device="cuda").to(t), i32([L]), i32([0, n]), i32([-1] + [0] * (n - 1)))
        for n, g, t in ((4, 1, torch.bfloat16), (24, 1, torch.bfloat16), (100, 2, torch.bfloat16), (20, 1, torch.float32))]
everything = i32([0, L + 128])
torch.cuda.synchronize()
def calls():
    ttv.kv4_write(k, v, cache, zero, everything, st)
    out = [ttv.tree_attn_kv4(q, cache, l, off, None, L, st, parents=par) for q, l, off, par in runs]
    return out + list(ttv.kv4_read(cache, zero, everything, st, rows=L + 128))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, calls())) and st.tolist() == [0]
print("the same")
"""


def test_first_calls_inside_a_capture():
    """A new process whose first calls are captured: what a launch asks of a kernel once is no stream operation."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]


def test_the_dense_attention_agrees_on_the_values_read_back():
    """Slots read back into a dense cache give spec_tree_attn the same keys and values."""
    rng = np.random.default_rng(18)
    L, n, H, D, cap = [90, 33], [20, 7], 2, 128, 115
    off = np.concatenate([[0], np.cumsum(n)])
    rec = random_records(rng, (2, H, cap), D)
    cache, st = torch.from_numpy(rec).cuda(), zeros_status(2)
    dense = torch.zeros((2, 2, H, cap, D), dtype=BF16, device="cuda")
    for b in range(2):
        keys = L[b] + n[b]
        ttv.kv4_read(cache[b:b + 1], i32([0]), i32([0, keys]), st[b:b + 1],
                     out=(dense[0, b].transpose(0, 1)[:keys], dense[1, b].transpose(0, 1)[:keys]))
    par = i32(sum((random_tree(rng, c) for c in n), []))
    q = torch.randn((off[-1], 8, D), device="cuda").to(BF16)
    a = ttv.tree_attn(q, dense[0], dense[1], i32(L), i32(off), None, max(L), st, parents=par)
    b = ttv.tree_attn_kv4(q, cache, i32(L), i32(off), None, max(L), st, parents=par)
    # both are within 2^-8 |o| + 2^-11 mean|v| of the exact result
    _, size, _, _ = kv4.tree_attn(q.float().cpu().numpy(), rec, L, off, par.cpu().numpy())
    assert (np.abs(a.double().cpu().numpy() - b.double().cpu().numpy()) <= 2.0 ** -6 * size).all()
    assert st.tolist() == [0, 0]


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_what_the_calls_do_not_cover():
    cache, st = ttv.make_kv4_cache(1, 2, 16, 128), zeros_status(1)
    rows = torch.zeros((4, 2, 128), dtype=BF16, device="cuda")
    off, start = i32([0, 4]), i32([0])
    with pytest.raises(ValueError):
        ttv.make_kv4_cache(1, 2, 16, 96)
    with pytest.raises(TypeError):
        ttv.kv4_write(rows.half(), rows.half(), cache, start, off, st)
    with pytest.raises(TypeError):
        ttv.kv4_write(rows, rows.float(), cache, start, off, st)
    with pytest.raises(ValueError):
        ttv.kv4_write(rows[:, :1], rows, cache, start, off, st)
    with pytest.raises(ValueError):
        ttv.kv4_write(rows.transpose(1, 2).contiguous().transpose(1, 2), rows, cache, start, off, st)
    with pytest.raises(TypeError):
        ttv.kv4_write(rows.cpu(), rows, cache, start, off, st)
    with pytest.raises(TypeError):
        ttv.kv4_write(rows, rows, cache, start.long(), off, st)
    with pytest.raises(ValueError):
        ttv.kv4_write(rows, rows, cache, start, off[:1], st)
    with pytest.raises(ValueError):
        ttv.kv4_write(rows, rows, cache[..., :100], start, off, st)
    with pytest.raises(ttv.SpecError):       # rows that start 2 bytes off a 16-byte boundary
        ttv.kv4_write(torch.zeros(4 * 256 + 1, dtype=BF16, device="cuda")[1:].view(4, 2, 128), rows, cache, start, off, st)
    with pytest.raises(ValueError):
        ttv.kv4_read(cache, start, off, st)
    with pytest.raises(ttv.SpecError):       # overlapping output rows
        ttv.kv4_read(cache, start, off, st, out=(rows[:1].expand(4, 2, 128), rows))
    q = torch.zeros((4, 4, 128), dtype=BF16, device="cuda")
    mask = torch.zeros((4, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ttv.tree_attn_kv4(q, cache, start, off, None, 0, st)
    with pytest.raises(ValueError):
        ttv.tree_attn_kv4(q[:, ::2], cache, start, off, mask, 0, st)
    with pytest.raises(TypeError):
        ttv.tree_attn_kv4(q.half(), cache, start, off, mask, 0, st)
    with pytest.raises(ttv.SpecError):
        ttv.tree_attn_kv4(torch.zeros((4, 3, 128), dtype=BF16, device="cuda"), cache, start, off, mask, 0, st)
    with pytest.raises(ttv.SpecError):
        ttv.tree_attn_kv4(q, cache, start, off, mask, 0, st, window=-1)
    with pytest.raises(ttv.SpecError):
        ttv.kv4_compact(cache, start, off, i32([[0, 1]]), i32([1]), st, new_prefix_lens=start)
    torch.cuda.synchronize()
    assert st.tolist() == [0]
