"""The paged calls through the module of csrc/marshal.cpp and through binding.py
alone: the same outputs, the same exceptions, and the module takes what it should."""
import contextlib

import numpy as np
import pytest
import torch

import token_tree_verification_gb300 as ttv
from test_gpu_paged import BF16, Cache, gpu, i32, zeros_status
from token_tree_verification_gb300 import binding

pytestmark = pytest.mark.gpu
F32 = torch.float32


def make(dtype, D=64):
    rng = np.random.default_rng(1)
    cache = Cache(rng, [40, 60], 2, 16, D, dtype, fill=0.5)
    q, k, v = (gpu(rng.standard_normal((15, h, D)), dtype) for h in (6, 2, 2))
    return dict(q=q, k=k, v=v, kp=cache.k, vp=cache.v, table=cache.block_table, lens=i32([20, 7]), off=i32([0, 5, 15]),
                st=zeros_status(2), rope=ttv.rope_table(32, 10000.0, "yarn", 2.0, original=16.0), depth=i32(range(15)),
                path=i32([[0, 2, 4], [0, 1, -1]]), acc=i32([2, 1]), par=i32([-1, 0, 1, 0, 3, -1, 0, 0, 1, 1, 2, 4, 5, 0, 8]))


CALLS = {
    "rope": lambda a, **kw: ttv.rope(a["q"], a["rope"], a["lens"], a["off"], a["st"], **kw),
    "write": lambda a, **kw: ttv.rope_write_paged(a["q"], a["k"], a["v"], a["kp"], a["vp"], a["table"], a["lens"], a["off"],
                                                  a["st"], a["rope"], **kw),
    "attn": lambda a, **kw: ttv.tree_attn_paged(a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["off"], a.get("mask"), 20,
                                                a["st"], **({"parents": a["par"]} | kw)),
    "compact": lambda a, **kw: ttv.kv_compact_paged(a["kp"], a["vp"], a["table"], a["lens"], a["off"], a["path"], a["acc"],
                                                    a["st"], **kw),
}
GOOD = [("rope", {}), ("rope", dict(interleaved=True)), ("rope", "depth"), ("write", {}), ("write", dict(interleaved=1)),
        ("write", "depth"), ("write", "start"), ("attn", {}), ("attn", dict(causal=True, parents=None)),
        ("attn", dict(softmax_scale=0.3)), ("attn", dict(softmax_scale=1)), ("compact", {})]


@contextlib.contextmanager
def without_module():
    kept, binding._marshal = binding._marshal, None
    try:
        yield
    finally:
        binding._marshal = kept


def outcome(name, a, kw):
    try:
        y = CALLS[name](a, **kw)
    except Exception as e:
        return type(e), str(e)
    return y, a["kp"].clone(), a["vp"].clone(), a["st"].clone()


def same(x, y):
    if isinstance(x, torch.Tensor):
        return x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and torch.equal(x, y)
    return x == y


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", range(len(GOOD)))
def test_the_module_takes_the_call(gpu_lib, dtype, case, monkeypatch):
    assert binding._marshal is not None, "csrc/marshal.cpp was not built"
    name, kw = GOOD[case]
    both = []
    for use in (True, False):
        a = make(dtype)
        args = {kw: a["depth"] if kw == "depth" else i32([3, 100])} if isinstance(kw, str) else kw
        if use:
            # binding.py's own way is closed: the module has to do it
            with monkeypatch.context() as m:
                m.setattr(binding, "_per_request", None)
                both.append(outcome(name, a, args))
        else:
            with without_module():
                both.append(outcome(name, a, args))
    for x, y in zip(*both):
        assert same(x, y)
    assert both[0][-1].eq(0).all()


BAD = [("rope", dict(q=lambda a: a["q"].half())), ("rope", dict(lens=lambda a: a["lens"][:1])), ("rope", dict(off=lambda a: a["off"].long())),
       ("rope", dict(q=lambda a: a["q"][0])), ("rope", dict(rope=lambda a: ttv.rope_table(128))),
       ("rope", dict(rope=lambda a: a["rope"]._replace(freqs=a["rope"].freqs.cpu()))), ("rope", dict(st=lambda a: a["st"].cpu())),
       ("rope", dict(q=lambda a: None)), ("write", dict(k=lambda a: a["k"][:, :1])), ("write", dict(v=lambda a: a["v"].float() + 0.0j)),
       ("write", dict(kp=lambda a: a["kp"].transpose(1, 2))), ("write", dict(table=lambda a: a["table"][:1])),
       ("write", dict(st=lambda a: i32([]), lens=lambda a: i32([]), off=lambda a: i32([0]), table=lambda a: a["table"][:0])),
       ("attn", dict(q=lambda a: a["q"][:, :5])), ("attn", dict(q=lambda a: a["q"][:, :, :32])), ("attn", dict(par=lambda a: None)),
       ("attn", dict(mask=lambda a: torch.zeros((3, 4), dtype=torch.int32, device="cuda"))),
       ("attn", dict(vp=lambda a: a["vp"][:3])), ("compact", dict(path=lambda a: a["path"].flatten())),
       ("compact", dict(acc=lambda a: a["acc"].float())), ("compact", dict(kp=lambda a: a["kp"].cpu()))]


@pytest.mark.parametrize("case", range(len(BAD)))
def test_what_the_module_does_not_take_ends_as_without_it(gpu_lib, case):
    name, change = BAD[case]
    both = []
    for use in (True, False):
        a = make(BF16)
        for key, f in change.items():
            a[key] = f(a)
        with contextlib.nullcontext() if use else without_module():
            both.append(outcome(name, a, {}))
    assert isinstance(both[0][0], type) and both[0] == both[1], both


def test_device_errors_are_the_same(gpu_lib):
    for use in (True, False):
        a = make(BF16)
        a["table"][1, 0] = 1000
        with contextlib.nullcontext() if use else without_module():
            for name in ("write", "attn"):
                a["st"].zero_()
                CALLS[name](a)
                assert a["st"].tolist() == [0, -14], (use, name)
