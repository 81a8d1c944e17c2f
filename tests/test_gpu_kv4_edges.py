"""The 4-bit cache's calls at the edges of what they take: scores and scales at
the ends of fp32, and the calls that a batch or a caller makes rarely."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import token_tree_verification_gb300 as ttv
from oracle import kv4
from test_gpu_kv4 import BF16, DTYPES, check_attn, i32, random_records, random_tree, zeros_status

pytestmark = pytest.mark.gpu


# Each form of the attention: up to 8, 16, 32 and 128 rows on a key.
FORMS = pytest.mark.parametrize("Hq,n", [(1, 7), (2, 8), (2, 15), (2, 40)], ids=["8", "16", "32", "128"])


@DTYPES
@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 24, 2.0 ** 26, 2.0 ** 29, 1e12, 1e25, 1e36])
def test_scores_of_any_size(dtype, Hq, n, D, size):
    """Scores so large that fp32 holds no fraction of them: the output lies between the values seen, and is
    the best key's value where that key leads by more than the scores can be off."""
    rng = np.random.default_rng(D + n)
    L = 900
    rec = random_records(rng, (1, 1, L + n + 2), D)
    rec[..., L + n:, :] = 255
    parents = random_tree(rng, n)
    q = torch.from_numpy((rng.standard_normal((n, Hq, D)) * size).astype(np.float32)).to(dtype)
    st = zeros_status(1)
    o = ttv.tree_attn_kv4(q.cuda(), torch.from_numpy(rec).cuda(), i32([L]), i32([0, n]), None, L, st, parents=i32(parents))
    got = o.double().cpu().numpy()
    assert st.tolist() == [0] and np.isfinite(got).all()
    k, v = kv4.values(rec[0, 0, :L + n], D)
    ok = kv4.sees(parents, L)[:, None, :]
    x, scale = q.double().numpy(), 1 / np.sqrt(D)
    s = np.where(ok, np.einsum("ngd,sd->ngs", x, k) * scale, -np.inf)
    big = np.where(ok, np.einsum("ngd,sd->ngs", np.abs(x), np.abs(k)) * scale, 0).max(-1)
    # A score is off by at most (2^-21 + D 2^-24) sum |q||k| (query halves, sums of D products in fp32), and
    # twice that by 2^-22 of itself (its rounding, and the reference's).  40 more make every other weight
    # less than e^-40 of the best key's, 900 of them together less than 2^-47.
    order = np.sort(s, -1)
    clear = order[..., -1] - order[..., -2] > 2 * (2.0 ** -20 + D * 2.0 ** -24) * big + 40
    assert clear.mean() > 0.5           # (the best two of 900 keys are seldom that close)
    best = v[s.argmax(-1)]
    # the weight enters the product as a half (2^-11, two of them 2^-22) and the sum as it is; then the output's rounding
    tol = (2.0 ** -11 + 2.0 ** -8 if dtype == BF16 else 2.0 ** -21) * np.abs(best) * 1.01 + 2.0 ** -47 * np.abs(v).max()
    assert (np.abs(got - best) <= tol)[clear].all()
    seen = np.broadcast_to(ok[:, 0, :, None], (n, L + n, D))
    low = np.where(seen, v[None], np.inf).min(1)[:, None]
    high = np.where(seen, v[None], -np.inf).max(1)[:, None]
    room = 2.0 ** -7 * np.abs(v).max()
    assert (got >= low - room).all() and (got <= high + room).all()


@DTYPES
@FORMS
@pytest.mark.parametrize("scale,size", [(1e-9, 1e-36), (1e-38, 1.0), (1e-42, 1e3), (1e-42, 1e-36)])
def test_scales_so_small_that_all_keys_weigh_the_same(dtype, Hq, n, scale, size):
    """The factor of a row's scores may fall below what fp32 holds; masked keys stay out."""
    rng = np.random.default_rng(n)
    L, D = [150, 0], 128
    off = [0, n, 2 * n]
    rec = random_records(rng, (2, 1, 200), D)
    parents = random_tree(rng, n) + random_tree(rng, n)
    q = torch.from_numpy((rng.standard_normal((2 * n, Hq, D)) * size).astype(np.float32)).to(dtype)
    check_attn(q, rec, L, off, parents, scale=scale)


@DTYPES
@FORMS
def test_a_query_with_an_infinity_gives_nan_in_its_row_alone(dtype, Hq, n):
    rng = np.random.default_rng(n)
    D, L = 128, 300
    rec = torch.from_numpy(random_records(rng, (1, 1, L + n), D)).cuda()
    q = torch.from_numpy(rng.standard_normal((n, Hq, D)).astype(np.float32)).to(dtype).cuda()
    par, off, st = i32(random_tree(rng, n)), i32([0, n]), zeros_status(1)
    ref = ttv.tree_attn_kv4(q, rec, i32([L]), off, None, L, st, parents=par)
    q[n // 2, 0, 5] = float("inf")
    got = ttv.tree_attn_kv4(q, rec, i32([L]), off, None, L, st, parents=par)
    assert torch.isnan(got[n // 2, 0]).all()
    got[n // 2, 0] = ref[n // 2, 0]
    assert torch.equal(got, ref) and st.tolist() == [0]


# 9 to 16 rows on a key.  152 units (a request's rows on one KV head) are not split on this GPU's 152 SMs, so a
# CTA takes all the tiles of 128 keys: 11 to 15 here.  Eight units are split.
LONG = [  # D, Hq, Hkv, prefixes, nodes
    (128, 38, 38, [1900, 1660, 1400, 1285], [16, 9, 12, 16]),       # 15, 14, 12 and 11 tiles
    (64, 38, 38, [1900, 1660, 1400, 1285], [9, 16, 11, 13]),
    (128, 114, 38, [1500, 1850, 1300, 1600], [5, 4, 5, 3]),         # three query heads on each key
    # one request with many more rows than the mean, an odd and an even number of tiles in each turn
    (128, 38, 38, [1600, 300, 1285, 20], [45, 1, 1, 2]), (64, 38, 38, [1600, 300, 1285, 20], [45, 1, 1, 2]),
    (128, 38, 38, [40, 1400, 900, 20], [3, 58, 1, 1]), (64, 38, 38, [40, 1400, 900, 20], [3, 58, 1, 1]),
    (128, 2, 2, [9000, 300, 2000, 20], [45, 1, 1, 2]), (64, 2, 2, [9000, 300, 2000, 20], [45, 1, 1, 2])]


@DTYPES
@pytest.mark.parametrize("D,Hq,Hkv,L,n", LONG)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1290, 300)], ids=["all", "window"])
def test_nine_to_sixteen_rows_over_many_tiles_and_turns(dtype, D, Hq, Hkv, L, n, window, sinks):
    rng = np.random.default_rng(D + Hq + n[0])
    off = np.concatenate([[0], np.cumsum(n)])
    assert 9 <= -(-off[-1] // len(n)) * (Hq // Hkv) <= 16
    rec = random_records(rng, (len(L), Hkv, max(a + b for a, b in zip(L, n)) + 3), D)
    for b, (a, c) in enumerate(zip(L, n)):
        rec[b, :, a + c:] = 255
    parents = sum((random_tree(rng, c) for c in n), [])
    q = torch.from_numpy((2 * rng.standard_normal((off[-1], Hq, D))).astype(np.float32)).to(dtype)
    check_attn(q, rec, L, off, parents, window, sinks)


WITHOUT_GETTERS = """
import torch
torch.cuda.init()
for owner, name in ((torch._C, "_cuda_getCurrentRawStream"), (torch._C._dynamo.guards, "_empty_strided_cuda")):
    if hasattr(owner, name):
        delattr(owner, name)
import token_tree_verification_gb300 as ttv
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
cache, st = ttv.make_kv4_cache(1, 2, 20, 64), i32(0)
k = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
side = torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(side):
    ttv.kv4_write(k, k, cache, i32(0), i32(0, 4), st)
    o = ttv.tree_attn_kv4(k[:1], cache, i32(3), i32(0, 1), None, 3, st, parents=i32(-1))
    new = ttv.kv4_compact(cache, i32(3), i32(0, 1), i32(0), i32(0), st)
    back, _ = ttv.kv4_read(cache, i32(0), i32(0, 4), st, rows=4)
torch.cuda.synchronize()
one = 6 * 0.171875          # 1 in the cache: 1/6 lies between the scales 0.15625 and 0.171875, nearer to the latter
assert (back == one).all() and (o == one).all() and new.item() == 4 and st.item() == 0
print("the same")
"""


def test_calls_without_the_private_getters_of_torch():
    r = subprocess.run([sys.executable, "-c", WITHOUT_GETTERS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]


@DTYPES
def test_outputs_are_tensors_as_torch_makes_them(dtype):
    """Under deterministic algorithms, what a call leaves of a new output is filled as torch fills it."""
    cache, st, D = ttv.make_kv4_cache(2, 2, 30, 128), zeros_status(2), 128
    q = torch.ones((6, 2, D), dtype=dtype, device="cuda")
    parents, off = i32([-1, 0, -1, 0, 9, 9]), i32([0, 2, 4])
    junk = [torch.ones(64 << 20, dtype=torch.uint8, device="cuda") for _ in range(3)]     # no NaN in what is reused
    del junk
    torch.use_deterministic_algorithms(True)
    try:
        k, v = ttv.kv4_read(cache, i32([0, 0]), off, st, rows=6, dtype=dtype)
        o = ttv.tree_attn_kv4(q, cache, i32([5, 5]), off, None, 5, st, parents=parents)
    finally:
        torch.use_deterministic_algorithms(False)
    for x in (k, v, o):       # two rows behind the last request
        assert torch.isnan(x[4:]).all() and torch.isfinite(x[:4]).all()
    assert st.tolist() == [0, 0]


class Busy:
    """Some milliseconds of copies, 2 GB each, queued on a stream."""

    def __init__(self):
        self.a, self.b = torch.zeros((2, 1 << 30), dtype=torch.uint8, device="cuda").unbind()

    def queue(self, stream, copies=60):
        with torch.cuda.stream(stream):
            for _ in range(copies):
                self.b.copy_(self.a)


def test_outputs_on_another_stream_beside_work_in_flight():
    """The caller's stream is busy with a tensor that it has dropped: the output of a call on another stream,
    which does not wait, is not that tensor's memory.  Nor is an output that the caller's stream still reads
    handed to the next call."""
    rng = np.random.default_rng(31)
    n, main, side, busy = 9000, torch.cuda.current_stream(), torch.cuda.Stream(), Busy()
    cache = torch.from_numpy(random_records(rng, (1, 8, n), 128)).cuda()
    start, off, st = i32([0]), i32([0, n]), zeros_status(1)
    q, lens, one, par = torch.ones((1, 8, 128), dtype=BF16, device="cuda"), i32([n - 1]), i32([0, 1]), i32([-1])
    want = ttv.kv4_read(cache, start, off, st, rows=n) + (ttv.tree_attn_kv4(q, cache, lens, one, None, n, st, parents=par),)
    calls = lambda: (ttv.kv4_read(cache, start, off, st, rows=n, stream=side)  # noqa: E731
                     + (ttv.tree_attn_kv4(q, cache, lens, one, None, n, st, parents=par, stream=side),))
    kept = [torch.empty_like(x) for x in want]
    for _ in range(3):
        dropped = [torch.full_like(x, 3.0) for x in want]
        torch.cuda.synchronize()
        busy.queue(main)
        for a, b in zip(kept, dropped):
            a.copy_(b)
        addresses = {x.data_ptr() for x in dropped}
        del dropped, b
        out = calls()
        assert not addresses & {x.data_ptr() for x in out}
        side.synchronize()
        assert not main.query()            # (the side stream's calls were done long before)
        torch.cuda.synchronize()
        assert all((x == 3.0).all() for x in kept)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    for _ in range(3):
        out = calls()
        main.wait_stream(side)
        busy.queue(main)
        for a, b in zip(kept, out):
            a.copy_(b)
        addresses = {x.data_ptr() for x in out}
        del out, b
        again = calls()
        assert not main.query() and not addresses & {x.data_ptr() for x in again}
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        del again
    assert st.tolist() == [0]


def test_outputs_dropped_while_their_call_is_under_way():
    """Work on the other stream keeps the calls from starting: what they will write is not given to anyone."""
    rng = np.random.default_rng(32)
    n, side, busy = 2000, torch.cuda.Stream(), Busy()
    cache = torch.from_numpy(random_records(rng, (1, 8, n), 128)).cuda()
    start, off, st = i32([0]), i32([0, n]), zeros_status(1)
    path, acc = i32([[0]]), i32([0])
    q, lens, one, par = torch.ones((1, 8, 128), dtype=BF16, device="cuda"), i32([n - 1]), i32([0, 1]), i32([-1])
    for turn in range(4):            # (the first loads the kernels that it launches, which takes its time)
        torch.cuda.synchronize()
        busy.queue(side)
        out = list(ttv.kv4_read(cache, start, off, st, rows=n, stream=side))
        out.append(ttv.tree_attn_kv4(q, cache, lens, one, None, n, st, parents=par, stream=side))
        out.append(ttv.kv4_compact(cache, lens, one, path, acc, st, stream=side))
        addresses = {x.data_ptr() for x in out}
        shapes = [(x.shape, x.dtype) for x in out]
        del out
        fresh = [torch.full(s, 5, dtype=t, device="cuda") for s, t in shapes]
        assert turn == 0 or not side.query()
        assert not addresses & {x.data_ptr() for x in fresh}
        torch.cuda.synchronize()
        assert all((x == 5).all() for x in fresh)
    assert st.tolist() == [0]


@DTYPES
@pytest.mark.parametrize("D", [64, 128])
def test_single_rows_and_heads_of_any_stride(dtype, D):
    """torch reports anything as the stride of a dimension of one, an odd one too."""
    rng = np.random.default_rng(D)
    x = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype).cuda()  # noqa: E731
    single = x(D, 1).t()[:, None, :]
    assert single.shape == (1, 1, D) and single.stride(0) == 1 and single.is_contiguous()
    one_row, one_head = x(3 * D + 3)[:3 * D].view(3, D).as_strided((1, 3, D), (5, D, 1)), x(7, D).as_strided((7, 1, D), (D, 3, 1))
    for rows in (single, one_row, one_head):
        T, H, _ = rows.shape
        cache, st = ttv.make_kv4_cache(1, H, 9, D), zeros_status(1)
        ttv.kv4_write(rows, rows, cache, i32([1]), i32([0, T]), st)
        want = np.zeros(cache.shape, np.uint8)
        kv4.write(want, rows.float().cpu().numpy(), rows.float().cpu().numpy(), [1], [0, T])
        np.testing.assert_array_equal(cache.cpu().numpy(), want)
        out = torch.full((2, T * H * D), 7.0, dtype=dtype, device="cuda")
        out = [y.as_strided((T, H, D), rows.stride(), y.storage_offset()) for y in out]
        ttv.kv4_read(cache, i32([1]), i32([0, T]), st, out=out)
        for got, ref in zip(out, kv4.read(want, D, [1], [0, T])):
            np.testing.assert_array_equal(got.double().cpu().numpy(), ref)
        assert st.tolist() == [0]


@DTYPES
@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [1e2, 1e4, 1e6, 1e12, 1e28])
@pytest.mark.parametrize("size", [2, 500])
def test_keys_far_below_the_others_come_first(dtype, Hq, n, D, far, size):
    """Runs of 256 keys whose scores are about -5000 x far, then 256 of ordinary ones, and so on: the softmax's
    reference has to come all the way up without a trace."""
    rng = np.random.default_rng(D + n)
    L = 9000
    rec = random_records(rng, (1, 1, L + n), D)
    low = (np.arange(L + n) % 512 < 256) & (np.arange(L + n) < L)
    rec[0, 0, :, 0] &= 0xF0                              # dimension 0 of the keys: 0, or -6 x 10240
    rec[0, 0, low, 0] |= 0xF
    rec[0, 0, low, D] = kv4.MAX_SCALE_BYTE
    rec[0, 0, low, 1:8] = 0                              # (the others of its group would be as large)
    rec[0, 0, low, 0] &= 0x0F
    parents = random_tree(rng, n)
    q = size * rng.standard_normal((n, Hq, D))
    q[..., 0] = far
    q = torch.from_numpy(q.astype(np.float32)).to(dtype)
    st = zeros_status(1)
    o = ttv.tree_attn_kv4(q.cuda(), torch.from_numpy(rec).cuda(), i32([L]), i32([0, n]), None, L, st, parents=i32(parents))
    got = o.double().cpu().numpy()
    k, v = kv4.values(rec[0, 0], D)
    x, scale = q.double().numpy(), 1 / np.sqrt(D)
    seen = kv4.sees(parents, L)[:, None, :]
    near = seen & ~low                                   # the others' weights are 0: e^-300000 and less
    s = np.where(near, np.einsum("ngd,sd->ngs", x, k) * scale, -np.inf)
    assert np.where(seen & low, np.einsum("ngd,sd->ngs", x, k) * scale, -np.inf).max() < s.max(-1).min() - 1e5
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    want, size = np.einsum("ngs,sd->ngd", p, v), np.einsum("ngs,sd->ngd", p, np.abs(v))
    # As for any attention, from the near keys alone: their dimension 0 is 0, so `far` is no part of their scores.
    # A query's elements beside it are halves of the row's scale: their smallest step is 2^-38 of the row's largest.
    big = np.where(near, np.einsum("ngd,sd->ngs", np.abs(x), np.abs(k)) * scale, 0).max(-1)[..., None]
    lost = 2.0 ** -38 * far * scale * np.where(near, np.abs(k).sum(-1), 0).max(-1)[..., None]
    delta = (2.0 ** -21 + D * 2.0 ** -24) * big + lost + 2.0 ** -20
    weight, last = (2.0 ** -11, 2.0 ** -8) if dtype == BF16 else (2.0 ** -22, 2.0 ** -24)
    reach = np.einsum("ngs,sd->ngd", np.broadcast_to(near, s.shape).astype(np.float64), np.abs(v))
    tol = size * (2 * delta + weight + 2.0 ** -18) + last * np.abs(want) * 1.01 + 2.0 ** -32 * reach
    assert st.tolist() == [0] and np.isfinite(got).all()
    if far <= 1e6:                       # (beyond, the elements beside `far` are lost, and the near keys' scores with them)
        assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
    else:
        top = np.where(near[..., None], np.abs(v)[None, None], 0).max((0, 1, 2))
        assert (np.abs(got) <= 1.01 * top).all()
