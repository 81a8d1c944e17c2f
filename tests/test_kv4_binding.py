"""The binding's own work on the host: what it needs of torch at import, and
whose memory the outputs of the 4-bit cache's calls are."""
import contextlib
import ctypes
import os
import subprocess
import sys
import types

import pytest
import torch

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


class FakeTensor:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, shape, dtype, made_on=None):
        self.shape, self.dtype, self.made_on, self.recorded = shape, dtype, made_on, []

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def data_ptr(self):
        return 4096

    def stride(self):
        return tuple(int(torch.Size(self.shape[i + 1:]).numel()) for i in range(len(self.shape)))

    def record_stream(self, stream):
        self.recorded.append(stream)


def i32(*shape):
    return FakeTensor(shape, torch.int32)


class FakeStream:
    def __init__(self, name):
        self.name, self.cuda_stream = name, 1


def test_outputs_of_a_call_on_another_stream_are_memory_of_that_stream(monkeypatch):
    """Allocated while it is current, so that the allocator orders them behind its work and not another's; kept
    from reuse until the caller's stream is done with them too."""
    from token_tree_verification_gb300 import binding
    main, side = FakeStream("main"), FakeStream("side")
    now = [main]

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_current_stream", lambda _: 1)
    monkeypatch.setattr(binding, "_empty", lambda shape, strides, dtype: FakeTensor(shape, dtype, now[-1].name))
    monkeypatch.setattr(binding, "_lib", types.SimpleNamespace(**{
        name: lambda *_: 0 for name in ("spec_kv4_read", "spec_tree_attn_kv4", "spec_kv4_compact")}))
    cache, q = FakeTensor((2, 4, 30, 144), torch.uint8), FakeTensor((6, 8, 128), torch.bfloat16)
    for s, made_on, others in ((None, "main", []), (side, "side", [main])):
        out = list(binding.kv4_read(cache, i32(2), i32(3), i32(2), rows=6, stream=s))
        out.append(binding.tree_attn_kv4(q, cache, i32(2), i32(3), None, 20, i32(2), parents=i32(6), stream=s))
        out.append(binding.kv4_compact(cache, i32(2), i32(3), i32(2, 4), i32(2), i32(2), stream=s))
        assert [x.made_on for x in out] == [made_on] * 4
        assert all(x.recorded == others for x in out)


@pytest.mark.parametrize("name", ["spec_kv4_write", "spec_kv4_read"])
def test_strides_between_single_rows_and_heads_are_not_looked_at(name):
    """What torch reports for a dimension of one may be anything."""
    from token_tree_verification_gb300 import binding, build
    build.build()
    fake = ctypes.c_void_p(0x1000)       # never dereferenced: T = 0 launches nothing

    def call(T, H, strides, dtype=1):
        return getattr(binding.load(), name)(fake, fake, dtype, 1, T, H, 128, *strides, fake, 8, fake, fake, fake, None)

    assert call(0, 2, (1, 128, -3, 128)) == 0
    assert call(0, 1, (1, 7, -3, -9)) == 0
    assert call(0, 2, (256, 1, 256, 128)) == -11 and call(0, 2, (256, -128, 256, 128)) == -2      # two heads


def test_numbers_beyond_a_c_int_are_limits_or_refused(monkeypatch):
    """ctypes would pass 2^32 + 5 as 5."""
    from token_tree_verification_gb300 import binding
    seen = {}
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_current_stream", lambda _: 1)
    monkeypatch.setattr(binding, "_lib", types.SimpleNamespace(
        spec_tree_attn_kv4=lambda *a: seen.update(max_prefix=a[10], window=a[16], sinks=a[17]) or 0,
        spec_kv4_write=lambda *a: 0))
    cache, q = FakeTensor((2, 4, 30, 144), torch.uint8), FakeTensor((6, 8, 128), torch.bfloat16)

    def attn(**kw):
        args = dict(max_prefix=20, window=0, sinks=0)
        args.update(kw)
        binding.tree_attn_kv4(q, cache, i32(2), i32(3), None, status=i32(2), parents=i32(6), o=q, **args)
        return seen["max_prefix"], seen["window"], seen["sinks"]

    top = 2 ** 31 - 1
    assert attn(max_prefix=2 ** 31, window=2 ** 32 + 5, sinks=2 ** 32) == (top, top, top)
    assert attn(max_prefix=top, window=7, sinks=3) == (top, 7, 3)
    assert attn(window=-1) == (20, -1, 0)          # (the library refuses it)
    with pytest.raises(ValueError, match="rows"):
        k = FakeTensor((2 ** 32 + 3, 4, 128), torch.bfloat16)
        binding.kv4_write(k, k, cache, i32(2), i32(3), i32(2))
    k = FakeTensor((6, 4, 128), torch.bfloat16)
    binding.kv4_write(k, k, cache, i32(2), i32(3), i32(2))
