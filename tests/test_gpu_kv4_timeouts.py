"""The failure path of the 4-bit attention on the GPU without a fault: the
kernels are built with waits that give up after a few looks, so that some run
out while the copies and products that they wait for are still under way.  A
call then returns, a request whose wait ran out reports SPEC_ERR_TIMEOUT, no row
is written but as without the failure, and the next call is served."""
import concurrent.futures as cf
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import token_tree_verification_gb300 as ttv
from test_gpu_kv4 import BF16, F32, i32, random_records, random_tree, zeros_status
from token_tree_verification_gb300 import binding, build

pytestmark = pytest.mark.gpu
POLLS = [0, 2, 20, 100, 1000]
SPEC_ERR_TIMEOUT = -9


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    """The attention's entry point, by the number of looks of a wait."""
    d = tmp_path_factory.mktemp("waits")
    sources = [s for s in build.sources() if os.path.basename(s).startswith("attn_kv4")]
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
        out[n] = ctypes.CDLL(so).spec_tree_attn_kv4
        out[n].argtypes, out[n].restype = binding.load().spec_tree_attn_kv4.argtypes, ctypes.c_int
    return out


FORMS = [  # dtype, query heads on each of two KV heads, nodes of each request
    (BF16, 1, [5, 8, 3]), (F32, 1, [5, 8, 3]), (F32, 2, [8, 5, 40]), (F32, 4, [16, 9, 30]), (BF16, 2, [7, 8, 3]),
    (BF16, 1, [40, 1, 1]), (BF16, 2, [15, 13, 60]), (BF16, 8, [20, 33, 128])]


@pytest.mark.parametrize("polls", POLLS)
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("D", [64, 128])
def test_waits_that_run_out_end_the_call(libs, polls, form, D):
    dtype, G, n = FORMS[form]
    rng = np.random.default_rng(form)
    L, H = [300, 9000, 40], 2
    off = np.concatenate([[0], np.cumsum(n)])
    T, S = int(off[-1]), max(L) + max(n)
    cache = torch.from_numpy(random_records(rng, (3, H, S), D)).cuda()
    q = torch.from_numpy(rng.standard_normal((T, H * G, D)).astype(np.float32)).to(dtype).cuda()
    lens, offs, par = i32(L), i32(off), i32(sum((random_tree(rng, c) for c in n), []))
    call = lambda st: ttv.tree_attn_kv4(q, cache, lens, offs, None, max(L), st, parents=par)  # noqa: E731
    ref = call(zeros_status(3))
    for _ in range(3):
        o, st = torch.full_like(ref, 9.0), zeros_status(3)
        rc = libs[polls](q.data_ptr(), cache.data_ptr(), o.data_ptr(), 1 if dtype is BF16 else 0, 3, T, H * G, H, D, S,
                         max(L), lens.data_ptr(), offs.data_ptr(), None, par.data_ptr(), 0.0, 0, 0, st.data_ptr(),
                         torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        codes = st.tolist()
        assert all(c in (0, SPEC_ERR_TIMEOUT) for c in codes)
        if polls == 0:
            assert codes == [SPEC_ERR_TIMEOUT] * 3
        for b, code in enumerate(codes):
            got, want = o[off[b]:off[b + 1]], ref[off[b]:off[b + 1]]
            same = (got == want).all(-1)
            assert (same | ((got == 9.0).all(-1) & (code != 0))).all()
            assert polls or not same.any()
    st = zeros_status(3)
    assert torch.equal(call(st), ref) and st.tolist() == [0, 0, 0]
