"""The failure path of the attention over pages on the GPU without a fault: the
kernel is built with waits that give up after a few looks, so that some run out
while the copies and products that they wait for are still under way.  A call
then returns, a request whose wait ran out reports SPEC_ERR_TIMEOUT, no row is
written but as without the failure, and the next call is served."""
import concurrent.futures as cf
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import token_tree_verification_gb300 as ttv
from test_gpu_paged import BF16, batch, i32, random_tree, zeros_status
from token_tree_verification_gb300 import binding, build

pytestmark = pytest.mark.gpu
POLLS = [0, 2, 20, 100, 1000]
SPEC_ERR_TIMEOUT = -9


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    """The attention's entry point, by the number of looks of a wait."""
    d = tmp_path_factory.mktemp("waits")
    sources = [s for s in build.sources() if os.path.basename(s).startswith("attn_paged")]
    jobs = [(n, s, str(d / f"{os.path.basename(s)[:-3]}_{n}.o")) for n in POLLS for s in sources]

    def compile_one(job):
        n, s, obj = job
        cmd = [build._nvcc(), *build.ARCH, *build.FLAGS, f"-DSPEC_WAIT_POLLS={n}", "-c", s, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr

    with cf.ThreadPoolExecutor(os.cpu_count()) as ex:
        list(ex.map(compile_one, jobs))
    out = {}
    for n in POLLS:
        so = str(d / f"attn_{n}.so")
        r = subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", so, *(o for m, _, o in jobs if m == n)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        out[n] = ctypes.CDLL(so).spec_tree_attn_paged
        out[n].argtypes, out[n].restype = binding.load().spec_tree_attn_paged.argtypes, ctypes.c_int
    return out


FORMS = [  # query heads on each of two KV heads, new rows and prefixes of each request, runs of tokens
    (1, [5, 8, 3], [300, 9000, 40], False), (4, [1, 1, 1], [4000, 130, 2000], False), (8, [20, 33, 128], [300, 900, 40], False),
    (2, [700, 0, 300], [100, 50, 1500], True)]


@pytest.mark.parametrize("polls", POLLS)
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("D", [64, 128])
def test_waits_that_run_out_end_the_call(libs, polls, form, D):
    G, n, L, causal = FORMS[form]
    rng = np.random.default_rng(form)
    q, cache, off = batch(rng, n, L, 2 * G, 2, 32, D, BF16)
    lens, offs, table = i32(L), i32(off), cache.block_table
    par = None if causal else i32(sum((random_tree(rng, c) for c in n), []))
    call = lambda st: ttv.tree_attn_paged(q, cache.k, cache.v, table, lens, offs, None, max(L), st, parents=par,  # noqa: E731
                                          causal=causal)
    ref = call(zeros_status(3))
    for _ in range(3):
        o, st = torch.full_like(ref, 9.0), zeros_status(3)
        rc = libs[polls](q.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(), o.data_ptr(), 1, 3, int(off[-1]), 2 * G, 2, D,
                         cache.total, 32, table.data_ptr(), table.shape[1], max(L), lens.data_ptr(), offs.data_ptr(), None,
                         None if causal else par.data_ptr(), int(causal), 0.0, st.data_ptr(),
                         torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        codes = st.tolist()
        assert all(c in (0, SPEC_ERR_TIMEOUT) for c in codes)
        for b, code in enumerate(codes):
            if polls == 0 and n[b]:
                assert code == SPEC_ERR_TIMEOUT
            got, want = o[off[b]:off[b + 1]], ref[off[b]:off[b + 1]]
            same = (got == want).all(-1)
            assert (same | ((got == 9.0).all(-1) & (code != 0))).all()
    st = zeros_status(3)
    assert torch.equal(call(st), ref) and st.tolist() == [0, 0, 0]


@pytest.mark.parametrize("polls", POLLS)
@pytest.mark.parametrize("D", [64, 128])
def test_waits_that_run_out_in_launches_for_many_requests(libs, polls, D):
    rng = np.random.default_rng(7)
    B = 150
    n, L = rng.integers(1, 9, B).tolist(), rng.integers(0, 300, B).tolist()
    q, cache, off = batch(rng, n, L, 4, 2, 16, D, BF16)
    lens, offs, table = i32(L), i32(off), cache.block_table
    call = lambda st: ttv.tree_attn_paged(q, cache.k, cache.v, table, lens, offs, None, 300, st, causal=True)  # noqa: E731
    ref = call(zeros_status(B))
    for _ in range(3):
        o, st = torch.full_like(ref, 9.0), zeros_status(B)
        rc = libs[polls](q.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(), o.data_ptr(), 1, B, int(off[-1]), 4, 2, D,
                         cache.total, 16, table.data_ptr(), table.shape[1], 300, lens.data_ptr(), offs.data_ptr(), None, None, 1,
                         0.0, st.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        codes = st.tolist()
        assert all(c in (0, SPEC_ERR_TIMEOUT) for c in codes)
        for b, code in enumerate(codes):
            assert polls > 0 or code == SPEC_ERR_TIMEOUT
            got, want = o[off[b]:off[b + 1]], ref[off[b]:off[b + 1]]
            assert ((got == want).all(-1) | ((got == 9.0).all(-1) & (code != 0))).all()
    st = zeros_status(B)
    assert torch.equal(call(st), ref) and st.eq(0).all()
