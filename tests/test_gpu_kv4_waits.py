"""The bounded wait of the 4-bit attention's roles, in a kernel of its own: a
barrier that nothing completes is given up after the stated number of tries,
which take the stated time; one that is complete is not waited for, and one that
another warp completes meanwhile is seen."""
import ctypes
import subprocess

import pytest
import torch

from token_tree_verification_gb300 import build

pytestmark = pytest.mark.gpu

SOURCE = """
#include "attn_kv4.cuh"
using namespace spec;
// out: {done, ns} of a wait for a phase that never ends, one that is over, and one that warp 1 ends after 2 ms
__global__ void waits(unsigned long long *out, uint32_t tries) {
  __shared__ __align__(8) uint64_t bar[3];
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_arrive(&bar[1]);
  __syncthreads();
  for (int i = 0; i < 3; ++i) {
    const uint64_t t0 = global_ns();
    if (warp == 0) {
      const bool done = mbar_sleep(smem_addr(&bar[i]), 0, tries);
      if (threadIdx.x == 0) {
        out[2 * i] = done;
        out[2 * i + 1] = global_ns() - t0;
      }
    } else if (i == 2 && threadIdx.x == 32) {
      while (global_ns() - t0 < 2000000) {}
      mbar_arrive(&bar[2]);
    }
    __syncthreads();
  }
}
extern "C" int run_waits(unsigned long long *out, unsigned tries, void *stream) {
  waits<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(out, tries);
  return cudaGetLastError();
}
extern "C" unsigned limit_tries() { return kSleepTries; }
extern "C" unsigned long long limit_ns() { return kWaitLimitNs; }
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    src, out = d / "waits.cu", d / "waits.so"
    src.write_text(SOURCE)
    cmd = [build._nvcc(), *build.ARCH, *build.FLAGS, "-I", build.CSRC, "-shared", "-o", str(out), str(src)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(out))
    lib.run_waits.argtypes = [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]
    lib.limit_ns.restype = ctypes.c_uint64
    return lib


@pytest.mark.parametrize("tries", [1000, 10000])
def test_a_wait_ends_after_its_tries_which_make_its_limit(run, tries):
    out = torch.zeros(6, dtype=torch.int64, device="cuda")
    assert run.run_waits(out.data_ptr(), tries, torch.cuda.current_stream().cuda_stream) == 0
    never, never_ns, over, over_ns, soon, soon_ns = out.tolist()
    assert never == 0
    assert run.limit_ns() <= never_ns / tries * run.limit_tries() <= 1.1 * 10_000 * run.limit_tries()
    assert over == 1 and over_ns < 1e6
    assert soon == 1 and 1.9e6 < soon_ns < 4e6
