"""Rotary frequencies (computed on the host) and the refusals of the rotary and
paged calls, which come before any work on a device."""
import ctypes
import math

import numpy as np
import pytest

import token_tree_verification_gb300 as ttv
from oracle import paged

P, F32, F64, I64 = ctypes.c_void_p, ctypes.c_float, ctypes.c_double, ctypes.c_int64
FAKE = P(0x1000)      # never dereferenced

@pytest.fixture(scope="module")
def lib():
    from token_tree_verification_gb300 import build, binding
    build.build()
    return binding.load()

@pytest.mark.parametrize("r,base", [(128, 10000.0), (64, 500000.0), (2, 10.0), (24, 1e6), (512, 10000.0)])
@pytest.mark.parametrize("scaling,factor,original,low,high", [
    ("none", 1.0, 0.0, 1.0, None), ("linear", 3.0, 0.0, 1.0, None), ("ntk", 8.0, 0.0, 1.0, None),
    ("yarn", 16.0, 4096.0, 1.0, None), ("yarn", 2.0, 64.0, 2.0, 5.0), ("yarn", 1.0, 4096.0, 1.0, 32.0),
    ("bands", 8.0, 8192.0, 1.0, None), ("bands", 4.0, 100.0, 3.0, 3.5)])
def test_frequencies(lib, r, base, scaling, factor, original, low, high):
    if scaling == "ntk" and r == 2:
        pytest.skip("refused, see below")
    table = ttv.rope_table(r, base, scaling, factor, original=original, low=low, high=high, device="cpu")
    theta, scale = paged.frequencies(r, base, scaling, factor, original, low, high)
    got = np.array(table.freqs.tolist(), dtype=np.float64) * (2 * math.pi / 2.0 ** 64)
    # a power, a few products and quotients, two exponents up to ln(1e6) apart in their rounding
    assert np.allclose(got, theta, rtol=64 * 2.0 ** -53, atol=2.0 ** -61)
    assert table.scale == np.float32(scale) and table.rotary_dim == r

def test_a_rotation_is_refused(lib):
    out, scale = (ctypes.c_uint64 * 256)(), F32()
    f = lambda r=64, base=10000.0, kind=0, factor=1.0, original=0.0, low=1.0, high=4.0, to=out: lib.spec_rope_table(  # noqa: E731
        r, F64(base), kind, F64(factor), F64(original), F64(low), F64(high), to, ctypes.byref(scale))
    assert f() == 0 and f(to=None) == -1
    assert f(r=0) == f(r=3) == f(r=514) == f(r=-2) == -2
    assert f(base=1.0) == f(base=math.nan) == f(base=math.inf) == -2
    assert f(kind=-1) == f(kind=5) == -2
    assert f(kind=1, factor=0.5) == f(kind=1, factor=math.nan) == f(kind=1, factor=math.inf) == -2
    assert f(r=2, kind=2, factor=2.0) == -2
    for kind in (3, 4):
        assert f(kind=kind, factor=2.0, original=0.0) == -2
        assert f(kind=kind, factor=2.0, original=100.0, low=4.0, high=4.0) == -2
        assert f(kind=kind, factor=2.0, original=100.0, low=0.0) == -2
        assert f(kind=kind, factor=2.0, original=100.0) == 0
    with pytest.raises(ValueError):
        ttv.rope_table(64, scaling="other", device="cpu")
    with pytest.raises(ValueError):
        ttv.rope_table(100000, device="cpu")
    with pytest.raises(ttv.SpecError):
        ttv.rope_table(64, base=0.0, device="cpu")

def test_rows_are_refused(lib):
    def rope(x=FAKE, y=FAKE, dtype=1, B=1, T=4, H=2, D=64, xs=(128, 64), ys=(128, 64), freqs=FAKE, r=64, scale=1.0, start=FAKE,
             offsets=FAKE, status=FAKE):
        return lib.spec_rope(x, y, dtype, B, T, H, D, *(I64(s) for s in xs + ys), freqs, r, F32(scale), 0, start, None,
                             offsets, status, None)
    assert rope(T=0, x=None, y=None) == 0              # nothing to do
    for name in ("x", "y", "freqs", "start", "offsets", "status"):
        assert rope(**{name: None}) == -1, name
    assert rope(dtype=2) == -3
    assert rope(B=0) == rope(T=-1) == rope(H=0) == rope(D=60) == rope(D=0) == rope(D=520) == -2
    assert rope(r=65) == rope(r=66) == rope(r=-2) == rope(scale=math.nan) == rope(scale=math.inf) == -2
    assert rope(xs=(-128, 64)) == rope(ys=(0, 64)) == rope(ys=(128, 0)) == -2
    assert rope(x=P(0x1001)) == rope(freqs=P(0x1004)) == -11

def test_writes_into_pages_are_refused(lib):
    def write(q=FAKE, q_out=FAKE, k=FAKE, v=FAKE, dtype=1, B=1, T=4, Hq=4, Hkv=2, D=64, qs=(256, 64), ks=(128, 64),
              vs=(128, 64), freqs=FAKE, r=64, pool=FAKE, pages=10, size=16, table=FAKE, width=4, lens=FAKE, offsets=FAKE,
              status=FAKE):
        return lib.spec_rope_write_paged(q, q_out, k, v, dtype, B, T, Hq, Hkv, D, *(I64(s) for s in qs + ks + vs), freqs, r,
                                         F32(1.0), 0, pool, pool, pages, size, table, width, lens, None, None, offsets,
                                         status, None)
    assert write(T=0) == 0
    for name in ("q", "q_out", "k", "v", "freqs", "pool", "table", "lens", "offsets", "status"):
        assert write(**{name: None}) == -1, name
    assert write(dtype=-1) == -3
    for bad in (dict(pages=0), dict(size=0), dict(size=4), dict(size=48), dict(size=8192), dict(width=0), dict(Hkv=0),
                dict(Hq=-1), dict(D=12), dict(r=128), dict(ks=(-1, 64)), dict(vs=(128, -64)), dict(qs=(-8, 64))):
        assert write(**bad) == -2, bad
    assert write(pool=P(0x1008)) == write(k=P(0x1001)) == -11

def test_attention_over_pages_is_refused(lib):
    def attn(q=FAKE, pool=FAKE, o=FAKE, dtype=1, B=1, T=4, Hq=4, Hkv=2, D=64, pages=10, size=16, table=FAKE, width=4,
             max_prefix=8, lens=FAKE, offsets=FAKE, mask=FAKE, parents=None, causal=0, status=FAKE):
        return lib.spec_tree_attn_paged(q, pool, pool, o, dtype, B, T, Hq, Hkv, D, pages, size, table, width, max_prefix, lens,
                                        offsets, mask, parents, causal, F32(0.0), status, None)
    assert attn(T=0) == 0
    for name in ("q", "pool", "o", "table", "lens", "offsets", "mask", "status"):
        assert attn(**{name: None}) == -1, name
    assert attn(dtype=3) == -3
    assert attn(causal=1) == attn(causal=1, mask=None, parents=FAKE) == -2
    for bad in (dict(pages=0), dict(size=24), dict(width=0), dict(B=0), dict(T=-1), dict(Hq=3), dict(Hkv=0),
                dict(Hq=258), dict(D=96), dict(max_prefix=-1), dict(Hkv=65536, Hq=65536),
                dict(causal=1, mask=None, T=2 ** 30)):
        assert attn(**bad) == -2, bad
    for name in ("q", "pool", "o", "mask"):
        assert attn(**{name: P(0x1008)}) == -11, name

def test_moves_within_pages_are_refused(lib):
    def move(pool=FAKE, dtype=1, B=1, Hkv=2, D=64, pages=10, size=16, table=FAKE, width=4, lens=FAKE, offsets=FAKE, path=FAKE,
             accept=FAKE, W=4, new=P(0x2000), status=FAKE):
        return lib.spec_kv_compact_paged(pool, pool, dtype, B, Hkv, D, pages, size, table, width, lens, offsets, path, accept, W,
                                         new, status, None)
    for name in ("pool", "table", "lens", "offsets", "path", "accept", "new", "status"):
        assert move(**{name: None}) == -1, name
    assert move(dtype=9) == -3 and move(pool=P(0x1004)) == -11
    for bad in (dict(W=0), dict(W=129), dict(B=0), dict(B=65536), dict(Hkv=0), dict(D=32), dict(size=17), dict(pages=-1),
                dict(width=0), dict(new=FAKE)):
        assert move(**bad) == -2, bad

def test_lengths_that_overlap_are_refused(lib):
    def move(old, new, B):
        return lib.spec_kv_compact_paged(FAKE, FAKE, 1, B, 2, 64, 10, 16, FAKE, 4, P(old), FAKE, FAKE, FAKE, 4, P(new), FAKE, None)
    for old, new, B in ((0x2000, 0x2004, 2), (0x2004, 0x2000, 2), (0x2000, 0x2000 + 4 * 99, 100)):
        assert move(old, new, B) == -2


def test_rows_beyond_the_grid_are_refused(lib):
    assert lib.spec_rope(FAKE, FAKE, 1, 1, 2 ** 31 - 1, 1, 8, I64(8), I64(8), I64(8), I64(8), FAKE, 8, F32(1.0), 0, FAKE, None,
                         FAKE, FAKE, None) == -2


def test_the_oracle_rotates_whole_and_quarter_turns():
    """Positions of quarter turns, by hand."""
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    theta = np.array([math.pi / 2, math.pi])
    assert np.allclose(paged.rotate(x, np.array([1]), theta)[0], [[[-3, -2, 1, -4]]])
    assert np.allclose(paged.rotate(x, np.array([1]), theta, interleaved=True)[0], [[[-2, 1, -3, -4]]])
    assert np.allclose(paged.rotate(x, np.array([4]), theta)[0], x)

def test_the_oracle_attends_like_a_dense_one():
    """Pages in any order give what a softmax over the slots in order gives."""

    rng = np.random.default_rng(0)
    L, parents, H, G, D, size = 21, np.array([-1, 0, 0, 1, 3]), 2, 2, 8, 8
    n = len(parents)
    k, v = rng.standard_normal((2, 1, H, 40, D))
    q = rng.standard_normal((n, H * G, D))
    table = np.array([[3, 0, 4, 1]])
    pools = []
    for x in (k, v):
        pool = np.full((5, H, size, D), np.nan)
        for i in range(4):
            pool[table[0, i]] = x[0, :, i * size:(i + 1) * size]
        pools.append(pool)
    got = paged.attn(q, *pools, table, [L], [0, n], parents)[0]
    see = paged.sees(n, L, parents)
    for i in range(n):
        for h in range(H * G):
            s = k[0, h // G, :L + n] @ q[i, h] / math.sqrt(D)
            w = np.exp(s) * see[i]
            assert np.allclose(got[i, h], w @ v[0, h // G, :L + n] / w.sum())



def test_the_module_of_the_host_work(lib):
    """Built and bound here too; without a GPU it leaves every call to binding.py."""
    import torch
    from token_tree_verification_gb300 import binding
    assert binding._marshal is not None
    x, one = torch.zeros((2, 3, 64)), torch.zeros(1, dtype=torch.int32)
    assert binding._marshal.rope(x, None, one, one, one, None, False) is None
    assert binding._marshal.kv_compact_paged(x, x, x, x, x, x, x, x) is None
    assert binding._marshal.tree_attn_paged(*[None] * 12) is None
    assert binding._marshal.rope_write_paged(1, 2) is None
    with pytest.raises(TypeError):
        binding._marshal.bind(1, 2, 3)
    with pytest.raises(ValueError):
        binding._marshal.bind(1, 2, 3, 0)
    with pytest.raises(TypeError):
        ttv.rope(x, None, one, one, one)


def _theta_exactly(r, base, scaling, factor, original, low, high):
    """Turns a position of each pair, to 60 digits, from the formulas (Python's decimal); the ramp's ends as in the oracle."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")
    base, factor, original, low, high = (Decimal(x) for x in (base, factor, original, low, high))
    if scaling == "ntk":
        base *= factor ** (Decimal(r) / (r - 2))
    if scaling == "yarn":
        d = [r * (original / (2 * pi * t)).ln() / (2 * base.ln()) for t in (high, low)]
        first, last = max(0, math.floor(d[0])), min(r - 1, math.ceil(d[1]))
    out = []
    for i in range(r // 2):
        t = base ** (Decimal(-2 * i) / r)
        keep = Decimal(1)
        if scaling == "linear":
            keep = Decimal(0)
        elif scaling == "yarn":
            keep = 1 - min(Decimal(1), max(Decimal(0), Decimal(i - first) / max(Decimal(last - first), Decimal(0.001))))
        elif scaling == "bands":
            keep = min(Decimal(1), max(Decimal(0), (original * t / (2 * pi) - low) / (high - low)))
        out.append((t * keep + t / factor * (1 - keep)) / (2 * pi))
    return out

@pytest.mark.parametrize("r,base", [(128, 10000.0), (64, 500000.0), (2, 10.0), (4, 1.001), (24, 1e6), (512, 10000.0), (512, 9e29), (256, 1.5)])
@pytest.mark.parametrize("scaling,factor,original,low,high", [
    ("none", 1.0, 1.0, 1.0, 4.0), ("linear", 3.0, 1.0, 1.0, 4.0), ("linear", 9e8, 1.0, 1.0, 4.0), ("ntk", 8.0, 1.0, 1.0, 4.0),
    ("ntk", 1.7e6, 1.0, 1.0, 4.0), ("yarn", 16.0, 4096.0, 1.0, 32.0), ("yarn", 2.3, 64.0, 2.0, 5.0), ("yarn", 1.0, 4096.0, 1.0, 32.0),
    ("bands", 8.0, 8192.0, 1.0, 4.0), ("bands", 4.1, 100.0, 3.0, 3.5)])
def test_frequencies_to_the_last_place(lib, r, base, scaling, factor, original, low, high):
    """What a position multiplies, up to 2^32 times: half a unit of 2^-64 turns, and the two-double sums' own error,
    some 2^-100 for each of 256 products (beside it a ramp's or band's quotient)."""
    if scaling == "ntk" and r == 2:
        pytest.skip("refused, see above")
    table = ttv.rope_table(r, base, scaling, factor, original=original, low=low, high=high, device="cpu")
    for i, turns in enumerate(_theta_exactly(r, base, scaling, factor, original, low, high)):
        assert abs(float(table.freqs[i].item() % 2 ** 64 - turns * 2 ** 64)) <= 0.5 + 2.0 ** -20, i


def test_more_requests_than_a_compaction_takes_are_refused(lib):
    """The dense and the 4-bit call, as the paged one above."""
    for B, rc in ((65536, -2), (2 ** 31 - 1, -2)):
        assert lib.spec_kv_compact(FAKE, FAKE, 1, B, 2, 64, 40, FAKE, FAKE, FAKE, FAKE, 4, P(0x2000), FAKE, None) == rc
        assert lib.spec_kv4_compact(FAKE, B, 2, 64, 40, FAKE, FAKE, FAKE, FAKE, 4, P(0x2000), FAKE, None) == rc


def test_lengths_written_over_those_that_are_read_are_refused(lib):
    """The dense and the 4-bit call: a request's heads read its length while one of them writes the new one."""
    for old, new, B in ((0x2000, 0x2000, 1), (0x2000, 0x2004, 2), (0x2004, 0x2000, 2), (0x2000, 0x2000 + 4 * 99, 100)):
        assert lib.spec_kv_compact(FAKE, FAKE, 1, B, 2, 64, 40, P(old), FAKE, FAKE, FAKE, 4, P(new), FAKE, None) == -2
        assert lib.spec_kv4_compact(FAKE, B, 2, 64, 40, P(old), FAKE, FAKE, FAKE, 4, P(new), FAKE, None) == -2
