"""What the 4-bit attention's launches keep of a kernel, in a host program of its
own that sees no GPU: a query that failed is asked again."""
import os
import subprocess

from token_tree_verification_gb300 import build

SOURCE = """
#include <cstdio>
#include "attn_kv4.cuh"
using namespace spec;
__global__ void kernel(int) {}
int main() {
  static KernelState state;
  const int n = clusters_at_once(kernel, 2, 128, 1024, 0, &state);
  printf("%d clusters, kept %d\\n", n, state.at_once[0][2].load());
  return 0;
}
"""


def test_a_failed_occupancy_query_is_not_kept(tmp_path):
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(SOURCE)
    cmd = [build._nvcc(), *build.ARCH, *build.FLAGS, "-I", build.CSRC, "-o", str(exe), str(src)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert (r.returncode, r.stdout) == (0, "0 clusters, kept 0\n"), r.stdout + r.stderr
