"""The bounds-checked build's tests on a paged cache: a page's place in the block table and a row's place in the
pool are looked at before the access, and one outside is recorded and skipped.  A kernel of a few lines calls them (the
entry points never form such places: they refuse the request before)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from token_tree_verification_gb300 import build

CODE = """
#include "paged.cuh"
__global__ void probe(spec::PageTable p, int i, long long row, long long n, int *out) {
  out[0] = p.page(0, i);
  out[1] = p.holds(row, n, 2, 1);
}
extern "C" int run(const int *table, int *status, int i, long long row, long long n, int *out, void *stream) {
  probe<<<1, 1, 0, (cudaStream_t)stream>>>(spec::PageTable{table, 4, 3, 4, status}, i, row, n, out);
  return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def probe(gpu_lib, tmp_path_factory):
    where = tmp_path_factory.mktemp("checked")
    src, out = where / "probe.cu", where / "probe.so"
    src.write_text(CODE)
    subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, "-DSPEC_CHECKED", "-I", build.CSRC, "-shared", str(src), "-o", str(out)],
                   check=True)
    lib = ctypes.CDLL(str(out))
    lib.run.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p]
    return lib


@pytest.mark.gpu
@pytest.mark.parametrize("i,row,n,page,there,codes", [
    (2, 95, 1, 1, 1, [0, 0]), (3, 0, 96, -1, 1, [0, 0]), (0, 88, 8, 2, 1, [0, 0]),           # an id outside the pool is no index
    (4, 0, 1, -1, 1, [-12, 0]), (-1, 0, 1, -1, 1, [-12, 0]), (-2 ** 31, 0, 1, -1, 1, [-12, 0]), (2 ** 31 - 1, 0, 1, -1, 1, [-12, 0]),
    (0, 96, 1, 2, 0, [0, -12]), (0, 89, 8, 2, 0, [0, -12]), (0, -1, 1, 2, 0, [0, -12]), (0, 2 ** 40, 1, 2, 0, [0, -12])])
def test_places_outside_are_recorded_and_skipped(probe, i, row, n, page, there, codes):
    """A table of four entries, a pool of three pages of 16 slots and two heads: 96 rows."""
    table = torch.tensor([2, 0, 1, 7], dtype=torch.int32, device="cuda")
    status, out = (torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2))
    assert probe.run(table.data_ptr(), status.data_ptr(), i, row, n, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert out.tolist() == [page, there] and status.tolist() == codes


def test_every_kernel_on_pages_asks():
    """Where a row's place in a pool is formed from a page, the pool is asked whether it holds it."""
    for name, places in (("rope.cu", 1), ("kv_compact_paged.cu", 2), ("attn_paged_f32.cu", 2)):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        assert len(re.findall(r"pages\.holds\(", text)) == places, name
        assert "__ldg(" not in "".join(line for line in text.splitlines() if "pages.table" in line), name
