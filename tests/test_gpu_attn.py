"""GPU steps A2-A3 (spec_tree_attn) against the oracle's dense masked
attention, within max|d| <= 1e-2 max|ref| and relative error <= 2e-2."""
import numpy as np
import pytest
import torch

import oracle
from parity import assert_attn_close, gpu_attn, oracle_attn_rows
from token_tree_verification_gb300 import synthetic

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["tcgen05", "mma"])
def kernel(request, monkeypatch):
    """Both bf16 implementations: the tcgen05 kernel (default) and the
    mma.sync kernel (selected through SPEC_TREE_ATTN_KERNEL=mma)."""
    if request.param == "mma":
        monkeypatch.setenv("SPEC_TREE_ATTN_KERNEL", "mma")
    else:
        monkeypatch.delenv("SPEC_TREE_ATTN_KERNEL", raising=False)
    return request.param


def full_oracle(w):
    return oracle.tree_attn(w.q.float().numpy(), w.k_cache.float().numpy(), w.v_cache.float().numpy(),
                            w.prefix_lens, w.offsets, w.parents)


def test_tiny_fp32(gpu_lib):
    w = synthetic.make_workload("tiny", seed=0)
    got, st = gpu_attn(w)
    assert (st == 0).all()
    assert_attn_close(got, full_oracle(w), "tiny fp32")


@pytest.mark.parametrize("D,Hq,Hkv,L,N,B", [
    (128, 4, 4, 0, 8, 1),        # empty prefix
    (128, 4, 4, 1, 1, 1),        # root only, one prefix key
    (128, 2, 2, 63, 7, 2),       # ragged tail inside a tile
    (128, 2, 2, 64, 64, 1),      # tree fills exactly one tile
    (64, 8, 2, 200, 33, 3),      # D = 64, G = 4, several requests
    (128, 16, 2, 129, 40, 2),    # G = 8: rows = 320 (5 row blocks)
    (128, 4, 2, 300, 128, 1),    # largest tree
    (64, 2, 1, 1000, 17, 2),     # many tiles, many splits
])
def test_bf16_shapes(gpu_lib, kernel, D, Hq, Hkv, L, N, B):
    w = synthetic.make_workload("llama70b_gqa", seed=D + Hq + L + N, B=B, Hq=Hq, Hkv=Hkv, D=D, L=L,
                                N=N, depth=min(5, N - 1), width=8 if N > 40 else 4, V=64)
    got, st = gpu_attn(w)
    assert (st == 0).all()
    assert_attn_close(got, full_oracle(w), f"D{D} Hq{Hq} Hkv{Hkv} L{L} N{N} B{B}")


def test_fp32_ragged(gpu_lib):
    w = synthetic.make_workload("tiny", seed=5, B=3, L=77, N=20, depth=4, width=4, Hq=8, Hkv=2, D=128)
    got, st = gpu_attn(w)
    assert (st == 0).all()
    assert_attn_close(got, full_oracle(w), "fp32 ragged")


def test_llama7b_full(gpu_lib, kernel):
    w = synthetic.make_workload("llama7b", seed=0, device="cuda")
    got, st = gpu_attn(w)
    assert (st == 0).all()
    rows = np.arange(w.T * w.Hq)
    ref = oracle_attn_rows(w, rows)
    assert_attn_close(got.reshape(-1, w.D), ref, "llama7b")


@pytest.mark.parametrize("name", ["dynamic", "llama70b_gqa", "long_chain", "long_tree"])
def test_large_configs_sampled(gpu_lib, kernel, name):
    w = synthetic.make_workload(name, seed=0, device="cuda")
    got, st = gpu_attn(w)
    assert (st == 0).all()
    rng = np.random.default_rng(1)
    n_rows = w.T * w.Hq
    rows = np.unique(np.concatenate([
        rng.integers(0, n_rows, 96),
        # last node of every request, first and last head
        (w.offsets[1:] - 1) * w.Hq, (w.offsets[1:] - 1) * w.Hq + w.Hq - 1, w.offsets[:-1] * w.Hq]))
    ref = oracle_attn_rows(w, rows)
    assert_attn_close(got.reshape(-1, w.D)[rows], ref, name)


@pytest.mark.parametrize("Hq,Hkv,N,width,depth", [
    (4, 4, 10, 3, 2),     # 10 rows: a packed block
    (16, 2, 40, 4, 3),    # G = 8, 320 rows: 128-row blocks, the last one partial
])
def test_nan_padding_never_leaks(gpu_lib, kernel, Hq, Hkv, N, width, depth):
    w = synthetic.make_workload("llama7b", seed=3, L=100, N=N, width=width, depth=depth, Hq=Hq,
                                Hkv=Hkv, V=64, S_cap=256, pad=float("nan"))
    got, st = gpu_attn(w)
    assert (st == 0).all()
    assert np.isfinite(got).all()
    assert_attn_close(got, full_oracle(w), f"nan padding Hq{Hq} Hkv{Hkv} N{N}")


def test_rescale_path(gpu_lib, kernel):
    """Scores whose running max grows by far more than 2^8 across tiles (the
    tcgen05 kernel then rescales the stored O), with an explicit scale."""
    w = synthetic.make_workload("llama7b", seed=6, L=700, N=24, width=4, depth=3, Hq=4, Hkv=2, V=64)
    ramp = torch.linspace(0.2, 3.0, w.S_cap).view(1, 1, -1, 1)
    w.k_cache = (w.k_cache.float() * ramp).to(torch.bfloat16)
    w.q = (w.q.float() * 4.0).to(torch.bfloat16)
    import token_tree_verification_gb300 as ttv
    from parity import dev
    status = torch.zeros(w.B, dtype=torch.int32, device="cuda")
    mask, _ = ttv.build_tree_mask(dev(w.parents, torch.int32), dev(w.offsets, torch.int32), status)
    o = ttv.tree_attn(w.q.cuda(), w.k_cache.cuda(), w.v_cache.cuda(), dev(w.prefix_lens, torch.int32),
                      dev(w.offsets, torch.int32), mask, int(w.prefix_lens.max()), status,
                      softmax_scale=0.5)
    torch.cuda.synchronize()
    assert (status.cpu().numpy() == 0).all()
    ref = oracle.tree_attn(w.q.float().numpy(), w.k_cache.float().numpy(), w.v_cache.float().numpy(),
                           w.prefix_lens, w.offsets, w.parents, scale=0.5)
    assert_attn_close(o.float().cpu().numpy(), ref, "rescale")


def test_device_errors(gpu_lib):
    w = synthetic.make_workload("llama7b", seed=4, B=3, L=100, N=10, width=3, depth=2, Hq=4, Hkv=4,
                                V=64, S_cap=128)
    pl = w.prefix_lens.copy()
    pl[1] = 125          # 125 + 10 > S_cap
    w2 = w
    w2.prefix_lens = pl
    o_before = torch.full_like(w.q, 7.0).cuda()
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    import token_tree_verification_gb300 as ttv
    from parity import dev
    mask, _ = ttv.build_tree_mask(dev(w.parents, torch.int32), dev(w.offsets, torch.int32), status)
    o = ttv.tree_attn(w.q.cuda(), w.k_cache.cuda(), w.v_cache.cuda(), dev(pl, torch.int32),
                      dev(w.offsets, torch.int32), mask, 125, status, o=o_before)
    torch.cuda.synchronize()
    assert status.cpu().tolist() == [0, -10, 0]
    lo, hi = w.offsets[1], w.offsets[2]
    assert (o[lo:hi].float() == 7.0).all()        # untouched
    assert not (o[: w.offsets[1]].float() == 7.0).all()


def gpu_attn_parents(w, status=None, max_ctas=0):
    """spec_tree_attn_ex with no mask array: the kernel builds every row's
    ancestor set from the parent array."""
    import token_tree_verification_gb300 as ttv
    from parity import dev
    if status is None:
        status = torch.zeros(w.B, dtype=torch.int32, device="cuda")
    o = ttv.tree_attn(w.q.cuda(), w.k_cache.cuda(), w.v_cache.cuda(), dev(w.prefix_lens, torch.int32),
                      dev(w.offsets, torch.int32), None, int(w.prefix_lens.max()), status,
                      max_ctas=max_ctas, parents=dev(w.parents, torch.int32))
    torch.cuda.synchronize()
    return o.float().cpu().numpy().astype(np.float64), status.cpu().numpy()


@pytest.mark.parametrize("name,kw", [
    ("tiny", dict(B=3, L=77, N=20, depth=4, width=4, Hq=8, Hkv=2, D=128)),        # fp32 kernel
    ("llama70b_gqa", dict(B=1, Hq=4, Hkv=4, D=128, L=0, N=8, depth=5, width=4, V=64)),
    ("llama70b_gqa", dict(B=3, Hq=8, Hkv=2, D=64, L=200, N=33, depth=5, width=4, V=64)),
    ("llama70b_gqa", dict(B=2, Hq=16, Hkv=2, D=128, L=129, N=40, depth=5, width=8, V=64)),
    ("llama70b_gqa", dict(B=1, Hq=4, Hkv=2, D=128, L=300, N=128, depth=5, width=8, V=64)),
])
def test_parents_path(gpu_lib, kernel, name, kw):
    """Masks built in the kernel from the parents: outputs bit-identical to
    the mask-array path (the same ancestor bits) and within tolerance of the
    oracle."""
    if name == "tiny" and kernel == "mma":
        pytest.skip("fp32 inputs take the fp32 kernel either way")
    w = synthetic.make_workload(name, seed=11, **kw)
    got_m, st_m = gpu_attn(w)
    got_p, st_p = gpu_attn_parents(w)
    assert (st_m == 0).all() and (st_p == 0).all()
    assert np.array_equal(got_m, got_p)
    assert_attn_close(got_p, full_oracle(w), f"parents {name} {kw}")


def test_parents_path_llama7b_step_launch(gpu_lib):
    """The 7B workload as the timed step launches it: parents, no mask array,
    the split plan for the SMs verification leaves.  Bit-identical to the
    mask-array launch with the same plan (another split count rounds the
    merge differently), and within tolerance of the oracle on every row."""
    import token_tree_verification_gb300 as ttv
    from parity import dev
    w = synthetic.make_workload("llama7b", seed=0, device="cuda")
    status = torch.zeros(w.B, dtype=torch.int32, device="cuda")
    mask, _ = ttv.build_tree_mask(dev(w.parents, torch.int32), dev(w.offsets, torch.int32), status)
    o_m = ttv.tree_attn(w.q.cuda(), w.k_cache.cuda(), w.v_cache.cuda(), dev(w.prefix_lens, torch.int32),
                        dev(w.offsets, torch.int32), mask, int(w.prefix_lens.max()), status, max_ctas=118)
    torch.cuda.synchronize()
    got_p, st = gpu_attn_parents(w, max_ctas=118)
    assert (st == 0).all() and (status.cpu().numpy() == 0).all()
    assert np.array_equal(o_m.float().cpu().numpy().astype(np.float64), got_p)
    ref = oracle_attn_rows(w, np.arange(w.T * w.Hq))
    assert_attn_close(got_p.reshape(-1, w.D), ref, "llama7b, step launch")


def test_parents_path_bad_parent(gpu_lib, kernel):
    """A parent that is not below its node is reported for its request only;
    the other requests' rows are unaffected."""
    w = synthetic.make_workload("llama70b_gqa", seed=12, B=3, Hq=4, Hkv=2, D=128, L=90, N=12,
                                depth=3, width=4, V=64)
    ref_good, _ = gpu_attn_parents(w)
    par = w.parents.copy()
    lo = w.offsets[1]
    par[lo + 5] = 7          # forward parent in request 1
    w.parents = par
    got, st = gpu_attn_parents(w)
    assert st.tolist() == [0, -5, 0]   # SPEC_ERR_BAD_PARENT
    for b in (0, 2):
        a, z = w.offsets[b], w.offsets[b + 1]
        assert np.array_equal(got[a:z], ref_good[a:z])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_requests_without_rows_of_their_own_report(gpu_lib, kernel, dtype):
    """A tree without nodes, offsets below zero and beyond the batch; rows of no sound request stay as they were."""
    import token_tree_verification_gb300 as ttv
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn((12, 2, 64), device="cuda").to(dtype)
    k, v = (torch.randn((3, 2, 40, 64), device="cuda").to(dtype) for _ in range(2))
    three = [-1, 0, 0, 1] * 3
    for offsets, parents, codes, kept in (
            ([0, 4, 4, 12], three[:4] + [-1, 0, 0, 1, 2, 2, 3, 0], [0, -4, 0], []), ([-1, 4, 8, 12], three, [-4, 0, 0], [0, 1, 2, 3]),
            ([0, 4, 8, 13], three, [0, 0, -4], [8, 9, 10, 11]), ([0, 4, -1, 12], three, [0, -4, -4], list(range(4, 12)))):
        status, o = i32(0, 0, 0), torch.full_like(q, 7.0)
        ttv.tree_attn(q, k, v, i32(20, 30, 5), i32(*offsets), None, 40, status, o=o, parents=i32(*parents))
        same = o.eq(7).flatten(1).all(1).tolist()
        assert status.tolist() == codes and [i for i in range(12) if same[i]] == kept, offsets


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("by_parents", [False, True])
def test_prefixes_and_offsets_whose_sums_pass_31_bits(gpu_lib, kernel, dtype, by_parents):
    """A prefix that passes 2^31 with its tree, and offsets whose difference does and looks like a few nodes: errors,
    and rows that stay as they were."""
    import token_tree_verification_gb300 as ttv
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn((12, 2, 64), device="cuda").to(dtype)
    k, v = (torch.randn((3, 2, 40, 64), device="cuda").to(dtype) for _ in range(2))
    parents = i32(*[-1, 0, 0, 1] * 3)
    mask, _ = ttv.build_tree_mask(parents, i32(0, 4, 8, 12), i32(0, 0, 0))

    def call(lens, offsets):
        status, o = i32(0, 0, 0), torch.full_like(q, 7.0)
        ttv.tree_attn(q, k, v, i32(*lens), i32(*offsets), None if by_parents else mask, 40, status, o=o,
                      parents=parents if by_parents else None)
        return o, status.tolist()

    good, status = call([20, 36, 5], [0, 4, 8, 12])
    assert status == [0, 0, 0]
    o, status = call([20, 2 ** 31 - 1, 5], [0, 4, 8, 12])
    assert status == [0, -10, 0] and o[4:8].eq(7).all() and torch.equal(o[:4], good[:4]) and torch.equal(o[8:], good[8:])
    assert call([2 ** 31 - 4, 37, 2 ** 31 - 2], [0, 4, 8, 12])[1] == [-10, -10, -10]
    o, status = call([20, 20, 20], [0, 2 ** 31 - 1, -2 ** 31 + 3, 12])
    assert status == [-4, -4, -4] and o.eq(7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,mine", [(300, 299), (300, 0), (128, 127), (129, 5)])
def test_hundreds_of_requests_without_rows_report(gpu_lib, kernel, dtype, B, mine):
    """One node in all, of request `mine`; every other request is a tree without nodes."""
    import token_tree_verification_gb300 as ttv
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q, v = torch.ones((1, 2, 64), device="cuda").to(dtype), torch.full((B, 1, 3, 64), 0.5, device="cuda").to(dtype)
    status = i32([0] * B)
    o = ttv.tree_attn(q, v, v, i32([2] * B), i32([0] * (mine + 1) + [1] * (B - mine)), None, 2, status, parents=i32([-1]))
    assert status.tolist() == [0 if b == mine else -4 for b in range(B)] and o.eq(0.5).all()
