"""The 4-bit cache's oracle against the format's definition, and the refusals
of its entry points (which precede every CUDA call)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import kv4


def exact_nearest(x, table):
    """Brute force in rational arithmetic: nearest entry, ties to the even index."""
    x = Fraction(float(x))
    d = [abs(x - Fraction(float(t))) for t in table]
    best = min(d)
    hits = [i for i, y in enumerate(d) if y == best]
    return next((i for i in hits if i % 2 == 0), hits[0])


def test_scales_and_codes_are_the_nearest_in_rational_arithmetic():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 64)) * np.exp(3 * rng.standard_normal((40, 1)))).astype(np.float32)
    # groups whose maximum sits on, and one float beside, a boundary between two scales
    edge = 6 * (kv4.SCALES[:-1] + kv4.SCALES[1:]) / 2
    for i, near in enumerate((None, np.inf, -np.inf)):
        col = edge.astype(np.float32)
        col = col if near is None else np.nextafter(col, np.float32(near))
        pick = col[rng.integers(0, len(col), 20)]
        x[10 * i:10 * i + 10, 0] = pick[:10]
        x[10 * i:10 * i + 10, 16] = -pick[10:]
    code, byte, finite = kv4.quantise(x)
    assert finite.all()
    for r in range(x.shape[0]):
        for g in range(4):
            grp = x[r, 16 * g:16 * g + 16]
            b = exact_nearest(np.abs(grp).max(), [6 * s for s in kv4.SCALES])
            assert byte[r, g] == b
            s = Fraction(float(kv4.SCALES[b]))
            for j, e in enumerate(grp):
                want = exact_nearest(abs(Fraction(float(e))) / s, kv4.CODES) if s else 0
                got = int(code[r, 16 * g + j])
                assert (got & 7) == want and (got >> 3) == int(np.signbit(e))


def test_values_survive_bf16_and_half_and_requantisation():
    rng = np.random.default_rng(1)
    rec = rng.integers(0, 256, (50, kv4.record_bytes(128)), dtype=np.uint8)
    rec[:, 128:] = rng.integers(0, kv4.MAX_SCALE_BYTE + 1, (50, 16))
    k, v = kv4.values(rec, 128)
    for x in (k, v):
        t = torch.from_numpy(x)
        assert torch.equal(t.to(torch.bfloat16).double(), t)
        assert torch.equal(t.half().double(), t)
    assert kv4.MAX_SCALE_BYTE == 226 and kv4.SCALES[-1] == 10240.0


def test_window_by_hand():
    # root, 1 and 2 below the root, 3 below 1: positions 4, 5, 5, 6 behind four prefix keys
    ok = kv4.sees([-1, 0, 0, 1], 4, window=3, sinks=1)
    want = [[1, 0, 1, 1, 1, 0, 0, 0], [1, 0, 0, 1, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0, 1, 0], [1, 0, 0, 0, 1, 1, 0, 1]]
    np.testing.assert_array_equal(ok, np.array(want, bool))
    # sinks inside the tree when the prefix is shorter than they are
    ok = kv4.sees([-1, 0, 1, 2], 1, window=1, sinks=2)
    np.testing.assert_array_equal(ok[3], np.array([1, 1, 0, 0, 1], bool))


def test_attention_equals_the_dense_oracle_without_a_window():
    rng = np.random.default_rng(2)
    B, H, G, D, S = 2, 2, 2, 64, 40
    rec = rng.integers(0, 256, (B, H, S, kv4.record_bytes(D)), dtype=np.uint8)
    rec[..., D:] = rng.integers(90, 110, rec[..., D:].shape)
    off, L = np.array([0, 5, 12], np.int32), np.array([9, 30], np.int32)
    par = np.array([-1, 0, 0, 1, 1, -1, 0, 1, 2, 0, 0, 4], np.int32)
    q = rng.standard_normal((12, H * G, D)).astype(np.float32)
    k, v = (x.astype(np.float32) for x in kv4.values(rec, D))
    ref = oracle.tree_attn(q, k, v, L, off, par)
    got, _, _, _ = kv4.tree_attn(q, rec, L, off, par)
    np.testing.assert_allclose(got.reshape(-1), np.asarray(ref).reshape(-1), rtol=1e-6, atol=1e-6)


@pytest.fixture(scope="module")
def lib():
    from token_tree_verification_gb300 import binding, build
    build.build()
    return binding.load()


def test_refusals_before_any_launch(lib):
    P = ctypes.c_void_p
    fake = P(0x1000)   # never dereferenced
    assert [lib.spec_kv4_record_bytes(d) for d in (64, 128, 96, 0, -1)] == [80, 144, 0, 0, 0]

    def rows(f, k=fake, v=fake, dtype=1, B=2, T=4, H=2, D=128, st=(256, 128, 256, 128), kv=fake, S=8, start=fake,
             off=fake, status=fake):
        return f(k, v, dtype, B, T, H, D, *st, kv, S, start, off, status, None)

    for f in (lib.spec_kv4_write, lib.spec_kv4_read):
        for name in ("k", "v", "kv", "start", "off", "status"):
            assert rows(f, **{name: None}) == -1, name
        assert rows(f, dtype=2) == -3
        for bad in (dict(B=0), dict(T=-1), dict(H=0), dict(D=96), dict(S=0), dict(st=(-256, 128, 256, 128))):
            assert rows(f, **bad) == -2, bad
        assert rows(f, k=P(0x1008)) == -11 and rows(f, kv=P(0x1001)) == -11
        assert rows(f, st=(260, 128, 256, 128)) == -11      # 520 bytes: not a multiple of 16
        assert rows(f, T=0) == 0                              # nothing to do
    assert rows(lib.spec_kv4_read, st=(0, 128, 256, 128)) == -2
    assert rows(lib.spec_kv4_read, st=(256, 128, 256, 0)) == -2

    def attn(q=fake, kv=fake, o=fake, dtype=1, B=1, T=4, Hq=4, H=2, D=128, S=64, mp=32, L=fake, off=fake, mask=fake,
             par=None, window=0, sinks=0, status=fake):
        return lib.spec_tree_attn_kv4(q, kv, o, dtype, B, T, Hq, H, D, S, mp, L, off, mask, par, 0.0, window, sinks,
                                      status, None)

    for name in ("q", "kv", "o", "L", "off", "mask", "status"):
        assert attn(**{name: None}) == -1, name
    assert attn(dtype=5) == -3
    for bad in (dict(B=0), dict(T=0), dict(T=129), dict(Hq=3), dict(Hq=258), dict(H=0), dict(D=80), dict(S=0),
                dict(mp=-1), dict(window=-1), dict(sinks=-1), dict(S=2 ** 31 - 1024), dict(B=32768, H=2),
                dict(B=2 ** 31 - 1, T=2 ** 31 - 1, H=1)):
        assert attn(**bad) == -2, bad
    for name in ("q", "kv", "o", "mask"):
        assert attn(**{name: P(0x1004)}) == -11, name

    def compact(kv=fake, B=1, H=2, D=128, S=64, L=fake, off=fake, path=fake, acc=fake, W=4, new=P(0x2000), status=fake):
        return lib.spec_kv4_compact(kv, B, H, D, S, L, off, path, acc, W, new, status, None)

    for name in ("kv", "L", "off", "path", "acc", "new", "status"):
        assert compact(**{name: None}) == -1, name
    for bad in (dict(B=0), dict(B=65536), dict(H=0), dict(D=32), dict(S=0), dict(W=0), dict(W=129), dict(new=fake)):
        assert compact(**bad) == -2, bad
    assert compact(kv=P(0x1008)) == -11
    assert lib.spec_status_string(-13).decode().startswith("SPEC_ERR_NONFINITE")
