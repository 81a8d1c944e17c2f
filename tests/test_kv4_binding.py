"""The package imports wherever the public parts of torch are there."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("missing", ["torch._C._cuda_getDevice", "torch._C._cuda_getCurrentRawStream",
                                     "torch._C._dynamo.guards._empty_strided_cuda"])
def test_the_package_imports_without_a_private_part_of_torch(missing):
    owner, name = missing.rsplit(".", 1)
    code = (f"import torch\nowner = {owner}\nif hasattr(owner, {name!r}):\n    delattr(owner, {name!r})\n"
            "import token_tree_verification_gb300 as ttv\nfrom token_tree_verification_gb300 import synthetic\n"
            "assert ttv.tree_attn and ttv.kv4_write and synthetic.make_workload\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
