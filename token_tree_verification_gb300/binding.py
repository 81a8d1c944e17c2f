"""ctypes binding of ``libspec_tree.so`` (declared in include/spec_tree.h).

Argument marshalling only: torch tensors are checked for device, dtype and
contiguity, and their device pointers plus the current CUDA stream are passed
to the C ABI.  Every step of the computation runs in the library's CUDA
kernels; if the library cannot be loaded the calls raise, there is no CPU
fallback.

The library launches on the current CUDA device, so a call's tensors must
live there (``torch.cuda.set_device`` or ``with torch.cuda.device(...)``
around calls on another GPU).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple

import torch

from . import build

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None
# The module of csrc/marshal.cpp once the library is loaded, where it was built (for
# this torch and Python): the paged calls go through it, and it leaves what is not as
# it should be (it then returns None) to the functions here.
_marshal = None

STATUS = {
    0: "SPEC_OK", -1: "SPEC_ERR_NULL", -2: "SPEC_ERR_SHAPE", -3: "SPEC_ERR_DTYPE",
    -4: "SPEC_ERR_TREE_TOO_LARGE", -5: "SPEC_ERR_BAD_PARENT", -6: "SPEC_ERR_TOKEN_RANGE",
    -7: "SPEC_ERR_WORKSPACE", -8: "SPEC_ERR_CUDA", -9: "SPEC_ERR_TIMEOUT",
    -10: "SPEC_ERR_PREFIX_RANGE", -11: "SPEC_ERR_ALIGNMENT", -12: "SPEC_ERR_INDEX",
    -13: "SPEC_ERR_NONFINITE", -14: "SPEC_ERR_PAGE",
}
SPEC_F32, SPEC_BF16 = 0, 1
MAX_TREE_NODES = 128


class SpecError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)}")


def lib_path() -> str:
    """The library ``load()`` opens: the bounds-checked build when the
    environment sets ``SPEC_TREE_CHECKED=1`` (built by ``build(checked=True)``),
    the normal one otherwise."""
    if os.environ.get("SPEC_TREE_CHECKED", "0") == "1":
        return os.path.join(_HERE, "libspec_tree_checked.so")
    return os.path.join(_HERE, "libspec_tree.so")


def load():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with token_tree_verification_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I, U64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t, ctypes.c_float
    lib.spec_build_tree_mask.argtypes = [P, P, I, I, P, P, P, P]
    lib.spec_build_tree_mask.restype = I
    lib.spec_tree_attn_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.spec_tree_attn_workspace_size.restype = SZ
    lib.spec_tree_attn.argtypes = [P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, F, P, SZ, P, P]
    lib.spec_tree_attn.restype = I
    lib.spec_tree_attn_ex.argtypes = [P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, F, P, SZ, I, P, P]
    lib.spec_tree_attn_ex.restype = I
    lib.spec_tree_verify_workspace_size.argtypes = [I, I, I]
    lib.spec_tree_verify_workspace_size.restype = SZ
    lib.spec_tree_verify.argtypes = [P, P, P, P, P, I, I, I, F, U64, P, P, P, P, I, P, SZ, P, P]
    lib.spec_tree_verify.restype = I
    lib.spec_tree_verify_top_p.argtypes = [P, P, P, P, P, I, I, I, F, F, U64, P, P, P, P, I, P, SZ, P, P]
    lib.spec_tree_verify_top_p.restype = I
    lib.spec_kv_compact.argtypes = [P, P, I, I, I, I, I, P, P, P, P, I, P, P, P]
    lib.spec_kv_compact.restype = I
    I64 = ctypes.c_int64
    lib.spec_kv4_record_bytes.argtypes = [I]
    lib.spec_kv4_record_bytes.restype = SZ
    lib.spec_kv4_write.argtypes = [P, P, I, I, I, I, I, I64, I64, I64, I64, P, I, P, P, P, P]
    lib.spec_kv4_write.restype = I
    lib.spec_kv4_read.argtypes = [P, P, I, I, I, I, I, I64, I64, I64, I64, P, I, P, P, P, P]
    lib.spec_kv4_read.restype = I
    lib.spec_kv4_compact.argtypes = [P, I, I, I, I, P, P, P, P, I, P, P, P]
    lib.spec_kv4_compact.restype = I
    lib.spec_tree_attn_kv4.argtypes = [P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, F, I, I, P, P]
    lib.spec_tree_attn_kv4.restype = I
    DBL = ctypes.c_double
    lib.spec_rope_table.argtypes = [I, DBL, I, DBL, DBL, DBL, DBL, P, P]
    lib.spec_rope_table.restype = I
    lib.spec_rope.argtypes = [P, P, I, I, I, I, I, I64, I64, I64, I64, P, I, F, I, P, P, P, P, P]
    lib.spec_rope.restype = I
    lib.spec_rope_write_paged.argtypes = [P, P, P, P, I, I, I, I, I, I, I64, I64, I64, I64, I64, I64, P, I, F, I,
                                          P, P, I, I, P, I, P, P, P, P, P, P]
    lib.spec_rope_write_paged.restype = I
    lib.spec_tree_attn_paged.argtypes = [P, P, P, P, I, I, I, I, I, I, I, I, P, I, I, P, P, P, P, I, F, P, P]
    lib.spec_tree_attn_paged.restype = I
    lib.spec_kv_compact_paged.argtypes = [P, P, I, I, I, I, I, I, P, I, P, P, P, P, I, P, P, P]
    lib.spec_kv_compact_paged.restype = I
    lib.spec_tree_expand.argtypes = [P, P, P, P, I, I, I, F, U64, P, P, P, P]
    lib.spec_tree_expand.restype = I
    lib.spec_tree_prune.argtypes = [P, P, P, P, I, I, P, P, P, P, P, P]
    lib.spec_tree_prune.restype = I
    lib.spec_tree_merge.argtypes = [P, P, P, P, P, P, I, I, I, P, P, P, P, P, P]
    lib.spec_tree_merge.restype = I
    lib.spec_philox_uniforms.argtypes = [U64, P, I, P, P]
    lib.spec_philox_uniforms.restype = I
    lib.spec_status_string.argtypes = [I]
    lib.spec_status_string.restype = ctypes.c_char_p
    lib.spec_build_checked.argtypes = []
    lib.spec_build_checked.restype = I
    _lib = lib
    _load_marshal(lib)
    return lib


def _load_marshal(lib):
    global _marshal
    _marshal = None
    try:
        path = build.marshal_path()
        if not os.path.exists(path):
            return
        loader = importlib.machinery.ExtensionFileLoader(f"{__package__}._marshal", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location(loader.name, path, loader=loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (lib.spec_rope, lib.spec_rope_write_paged, lib.spec_tree_attn_paged,
                                                        lib.spec_kv_compact_paged)))
        _marshal = module
    except (ImportError, OSError):
        pass


def status_string(code: int) -> str:
    try:
        return load().spec_status_string(int(code)).decode()
    except Exception:  # library absent: fall back to the name table
        return STATUS.get(int(code), f"status {code}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _check(code: int, where: str):
    if code != 0:
        raise SpecError(code, where)


def build_tree_mask(parents, offsets, status, mask=None, depth=None, stream=None):
    """Step A1.  parents [T] int32, offsets [B+1] int32, status [B] int32 (zeroed
    by the caller).  Returns (mask [T, 4] int32 view of the uint32 bits, depth [T])."""
    lib = load()
    _dev(parents, torch.int32, "parents")
    _dev(offsets, torch.int32, "offsets")
    _dev(status, torch.int32, "status")
    T, B = parents.numel(), offsets.numel() - 1
    if mask is None:
        mask = torch.empty((T, 4), dtype=torch.int32, device=parents.device)
    if depth is None:
        depth = torch.empty(T, dtype=torch.int32, device=parents.device)
    _check(lib.spec_build_tree_mask(_ptr(parents), _ptr(offsets), B, T, _ptr(mask), _ptr(depth),
                                    _ptr(status), _stream(stream)), "spec_build_tree_mask")
    return mask, depth


def tree_attn_workspace_size(B, T, Hq, Hkv, D, max_prefix) -> int:
    return int(load().spec_tree_attn_workspace_size(B, T, Hq, Hkv, D, max_prefix))


def tree_attn(q, k_cache, v_cache, prefix_lens, offsets, mask, max_prefix, status, o=None,
              softmax_scale: float = 0.0, workspace=None, stream=None, max_ctas: int = 0,
              parents=None):
    """Steps A2-A3.  q [T, Hq, D]; k_cache, v_cache [B, Hkv, S_cap, D]; bf16 or fp32.
    ``max_ctas`` > 0 plans the launch for that many resident CTAs, leaving
    the other SMs to concurrent work; with ``mask=None`` the kernel builds
    every row's ancestor set from ``parents`` (both spec_tree_attn_ex)."""
    lib = load()
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError("q must be bfloat16 or float32")
    _dev(q, dt, "q")
    _dev(k_cache, dt, "k_cache")
    _dev(v_cache, dt, "v_cache")
    _dev(prefix_lens, torch.int32, "prefix_lens")
    _dev(offsets, torch.int32, "offsets")
    if mask is None:
        if parents is None:
            raise ValueError("tree_attn needs a mask or the parent array")
        _dev(parents, torch.int32, "parents")
    else:
        _dev(mask, torch.int32, "mask")
    _dev(status, torch.int32, "status")
    T, Hq, D = q.shape
    B, Hkv, S_cap, D2 = k_cache.shape
    if D2 != D or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("q / k_cache / v_cache shapes disagree")
    if o is None:
        o = torch.empty_like(q)
    ws_need = tree_attn_workspace_size(B, T, Hq, Hkv, D, max_prefix)
    if ws_need and workspace is None:
        workspace = torch.zeros(ws_need, dtype=torch.uint8, device=q.device)
    _check(lib.spec_tree_attn_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o),
                                 SPEC_BF16 if dt == torch.bfloat16 else SPEC_F32, B, T, Hq, Hkv, D,
                                 S_cap, int(max_prefix), _ptr(prefix_lens), _ptr(offsets),
                                 _ptr(mask), _ptr(parents) if mask is None else None,
                                 float(softmax_scale), _ptr(workspace),
                                 0 if workspace is None else workspace.numel(), int(max_ctas),
                                 _ptr(status), _stream(stream)), "spec_tree_attn_ex")
    return o


def tree_verify_workspace_size(B, T, V) -> int:
    return int(load().spec_tree_verify_workspace_size(B, T, V))


def make_verify_workspace(B, T, V, device="cuda"):
    """A zero-filled verification workspace (reusable across calls on one stream)."""
    return torch.zeros(tree_verify_workspace_size(B, T, V), dtype=torch.uint8, device=device)


def tree_verify(target_logits, draft_logits, tokens, parents, offsets, temperature: float,
                seed: int, max_depth_plus1: int, status, workspace, outputs=None, stream=None,
                top_p: float = 1.0):
    """Steps V1-V4 (top_p < 1: on the top_p nucleus of p and of q).  Returns
    dict(accept_len, path_nodes, out_tokens, near_ties) of device tensors."""
    lib = load()
    _dev(target_logits, torch.float32, "target_logits")
    if draft_logits is not None:
        _dev(draft_logits, torch.float32, "draft_logits")
    _dev(tokens, torch.int32, "tokens")
    _dev(parents, torch.int32, "parents")
    _dev(offsets, torch.int32, "offsets")
    _dev(status, torch.int32, "status")
    _dev(workspace, torch.uint8, "workspace")
    T, V = target_logits.shape
    B = offsets.numel() - 1
    W = int(max_depth_plus1)
    dev = target_logits.device
    if outputs is None:
        outputs = dict(
            accept_len=torch.empty(B, dtype=torch.int32, device=dev),
            path_nodes=torch.empty((B, W), dtype=torch.int32, device=dev),
            out_tokens=torch.empty((B, W), dtype=torch.int32, device=dev),
            near_ties=torch.empty(B, dtype=torch.int32, device=dev),
        )
    if top_p >= 1.0:
        _check(lib.spec_tree_verify(_ptr(target_logits), _ptr(draft_logits), _ptr(tokens),
                                    _ptr(parents), _ptr(offsets), B, T, V, float(temperature),
                                    int(seed) & (2**64 - 1), _ptr(outputs["accept_len"]),
                                    _ptr(outputs["path_nodes"]), _ptr(outputs["out_tokens"]),
                                    _ptr(outputs["near_ties"]), W, _ptr(workspace),
                                    workspace.numel(), _ptr(status), _stream(stream)),
               "spec_tree_verify")
        return outputs
    _check(lib.spec_tree_verify_top_p(_ptr(target_logits), _ptr(draft_logits), _ptr(tokens),
                                      _ptr(parents), _ptr(offsets), B, T, V, float(temperature),
                                      float(top_p), int(seed) & (2**64 - 1),
                                      _ptr(outputs["accept_len"]), _ptr(outputs["path_nodes"]),
                                      _ptr(outputs["out_tokens"]), _ptr(outputs["near_ties"]), W,
                                      _ptr(workspace), workspace.numel(), _ptr(status),
                                      _stream(stream)), "spec_tree_verify_top_p")
    return outputs


def kv_compact(k_cache, v_cache, prefix_lens, offsets, path_nodes, accept_len, status,
               new_prefix_lens=None, stream=None):
    """Depth-first KV-cache update after verification (in place).  Returns the
    new prefix lengths (device int32 [B])."""
    lib = load()
    if k_cache.dtype != v_cache.dtype or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must match")
    dt = {torch.bfloat16: SPEC_BF16, torch.float32: SPEC_F32}.get(k_cache.dtype)
    if dt is None:
        raise ValueError(f"unsupported cache dtype {k_cache.dtype}")
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _dev(t, k_cache.dtype, name)
    for t, name in ((prefix_lens, "prefix_lens"), (offsets, "offsets"), (path_nodes, "path_nodes"),
                    (accept_len, "accept_len"), (status, "status")):
        _dev(t, torch.int32, name)
    B, H, S_cap, D = k_cache.shape
    W = path_nodes.shape[-1]
    if new_prefix_lens is None:
        new_prefix_lens = torch.empty(B, dtype=torch.int32, device=k_cache.device)
    _check(lib.spec_kv_compact(_ptr(k_cache), _ptr(v_cache), dt, B, H, D, S_cap, _ptr(prefix_lens),
                               _ptr(offsets), _ptr(path_nodes), _ptr(accept_len), W,
                               _ptr(new_prefix_lens), _ptr(status), _stream(stream)),
           "spec_kv_compact")
    return new_prefix_lens


# ---------------------------------------------------------------- 4-bit cache
_KV4_DIMS = {144: 128, 80: 64}     # bytes of a slot record -> head dimension
_U8, _I32 = torch.uint8, torch.int32
# Parts of torch that are not public, used where they are there: the getters of the
# current device and stream, and a new tensor without the dispatcher (beside a
# launch 1.6 us of host time against 4.2 on a Grace core, an output of a call whose
# kernels take a few microseconds).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)
_empty_cuda = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)
_deterministic = torch.are_deterministic_algorithms_enabled      # torch then fills new tensors


def _empty(shape, strides, dtype):
    """A new tensor on the current device."""
    if _empty_cuda is None or _deterministic():
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")
    return _empty_cuda(shape, strides, dtype)


def _new(stream, shape, strides, dtype):
    """A new output of a call on ``stream`` (None: the current one).  It is memory
    of that stream, so that nothing else in flight still uses what the call
    writes, and once dropped it waits for the current stream's work too, which
    may read it."""
    if stream is None:
        return _empty(shape, strides, dtype)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = _empty(shape, strides, dtype)
    t.record_stream(current)
    return t


# The library takes C ints, to which ctypes cuts a number without a word.  What
# limits something may be any number; what counts rows may not.
_INT_MAX = 2 ** 31 - 1
_DTYPES = {torch.bfloat16: SPEC_BF16, torch.float32: SPEC_F32}


def kv4_record_bytes(D: int) -> int:
    """Bytes of one slot (key and value of one KV head) of a 4-bit cache, 0 for
    a head dimension it does not cover."""
    return int(load().spec_kv4_record_bytes(int(D)))


def make_kv4_cache(B, Hkv, S_cap, D, device="cuda"):
    """An empty 4-bit cache: uint8 [B, Hkv, S_cap, kv4_record_bytes(D)]."""
    R = kv4_record_bytes(D)
    if R == 0:
        raise ValueError(f"a 4-bit cache holds head dimensions 64 and 128, not {D}")
    return torch.zeros((B, Hkv, S_cap, R), dtype=torch.uint8, device=device)


def _kv4_cache(kv_cache):
    """Checks a 4-bit cache; returns (device index, B, Hkv, S_cap, D)."""
    index, shape = kv_cache.get_device(), kv_cache.shape
    D = _KV4_DIMS.get(shape[3]) if len(shape) == 4 else None
    if D is None or kv_cache.dtype is not _U8 or index != _current_device() or not kv_cache.is_contiguous():
        raise _not_a_cache(kv_cache, index)
    return index, shape[0], shape[1], shape[2], D


def _not_a_cache(kv_cache, index):
    if index < 0 or kv_cache.dtype is not _U8:
        return TypeError(f"kv_cache must be a CUDA tensor of torch.uint8, got {kv_cache.dtype} on {kv_cache.device}")
    if index != _current_device():
        return ValueError(f"kv_cache is on cuda:{index}, the current device is cuda:{_current_device()}")
    return ValueError("kv_cache must be contiguous [B, Hkv, S_cap, kv4_record_bytes(D)]")


def _not_i32(index, n, t, name):
    """The error of a tensor that is not n contiguous int32 on the device."""
    if t.dtype is not torch.int32 or t.get_device() != index:
        return TypeError(f"{name} must be torch.int32 on cuda:{index}, got {t.dtype} on {t.device}")
    return ValueError(f"{name} must be contiguous with {n} elements, got {tuple(t.shape)}")


def _i32(index, n, t, name):
    """The pointer of a device array of n int32."""
    if t.dtype is _I32 and t.get_device() == index and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    raise _not_i32(index, n, t, name)


def _per_request(index, B, first, offsets, status, name):
    """The pointers of the arrays that every call takes: B int32, the B + 1
    offsets and the B status words."""
    if (first.dtype is _I32 and offsets.dtype is _I32 and status.dtype is _I32
            and first.get_device() == offsets.get_device() == status.get_device() == index
            and first.numel() == status.numel() == B and offsets.numel() == B + 1
            and first.is_contiguous() and offsets.is_contiguous() and status.is_contiguous()):
        return first.data_ptr(), offsets.data_ptr(), status.data_ptr()
    return _i32(index, B, first, name), _i32(index, B + 1, offsets, "offsets"), _i32(index, B, status, "status")


def _dense_rows(index, t, T, Hkv, D, name):
    """Checks dense rows; returns their strides."""
    if t.get_device() != index:
        raise TypeError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.shape == (T, Hkv, D):
        row, head, one = t.stride()
        if one == 1 and T <= _INT_MAX:
            return row, head
    if T > _INT_MAX:
        raise ValueError(f"{name} may have {_INT_MAX} rows, not {T}")
    raise ValueError(f"{name} must be [{T}, {Hkv}, {D}] with its last dimension contiguous")


def kv4_write(k, v, kv_cache, start, offsets, status, stream=None):
    """Quantises dense rows into the 4-bit cache.  k, v [T, Hkv, D] (bf16 or
    fp32; rows and heads at any 16-byte stride); request b's rows
    offsets[b] .. offsets[b+1] go to slots start[b] and up."""
    lib = _lib or load()
    index, B, Hkv, S_cap, D = _kv4_cache(kv_cache)
    dt = _DTYPES.get(k.dtype)
    if dt is None or v.dtype is not k.dtype:
        raise TypeError("k and v must both be bfloat16 or float32")
    T = k.shape[0]
    ks0, ks1 = _dense_rows(index, k, T, Hkv, D, "k")
    vs0, vs1 = _dense_rows(index, v, T, Hkv, D, "v")
    start, offsets, status = _per_request(index, B, start, offsets, status, "start")
    rc = lib.spec_kv4_write(k.data_ptr(), v.data_ptr(), dt, B, T, Hkv, D, ks0, ks1, vs0, vs1, kv_cache.data_ptr(),
                            S_cap, start, offsets, status,
                            _current_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SpecError(rc, "spec_kv4_write")


def kv4_read(kv_cache, start, offsets, status, rows=None, dtype=torch.bfloat16, out=None, stream=None):
    """Reads slots of the 4-bit cache back as dense rows, the inverse of
    kv4_write: the first ``rows`` rows (offsets[-1] of them), or into
    ``out`` = (k, v), whose rows behind the last request stay as they are.
    Returns (k, v) [rows, Hkv, D]."""
    lib = _lib or load()
    index, B, Hkv, S_cap, D = _kv4_cache(kv_cache)
    if out is None:
        if rows is None:
            raise ValueError("kv4_read needs the number of rows, or out")
        T, ks0, ks1 = rows, Hkv * D, D
        vs0, vs1 = ks0, ks1
        k = _new(stream, (T, Hkv, D), (ks0, ks1, 1), dtype)
        v = _new(stream, (T, Hkv, D), (ks0, ks1, 1), dtype)
    else:
        k, v = out
        T = k.shape[0]
        ks0, ks1 = _dense_rows(index, k, T, Hkv, D, "k")
        vs0, vs1 = _dense_rows(index, v, T, Hkv, D, "v")
    dt = _DTYPES.get(k.dtype)
    if dt is None or v.dtype is not k.dtype:
        raise TypeError("rows are read as bfloat16 or float32")
    start, offsets, status = _per_request(index, B, start, offsets, status, "start")
    rc = lib.spec_kv4_read(k.data_ptr(), v.data_ptr(), dt, B, T, Hkv, D, ks0, ks1, vs0, vs1, kv_cache.data_ptr(),
                           S_cap, start, offsets, status,
                           _current_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SpecError(rc, "spec_kv4_read")
    return k, v


def kv4_compact(kv_cache, prefix_lens, offsets, path_nodes, accept_len, status,
                new_prefix_lens=None, stream=None):
    """kv_compact on a 4-bit cache (in place; records move as they are).
    Returns the new prefix lengths (device int32 [B])."""
    lib = _lib or load()
    index, B, Hkv, S_cap, D = _kv4_cache(kv_cache)
    W = path_nodes.shape[-1]
    if new_prefix_lens is None:
        new_prefix_lens = _new(stream, (B,), (1,), _I32)
    prefix, offsets, status = _per_request(index, B, prefix_lens, offsets, status, "prefix_lens")
    rc = lib.spec_kv4_compact(kv_cache.data_ptr(), B, Hkv, D, S_cap, prefix, offsets,
                              _i32(index, B * W, path_nodes, "path_nodes"),
                              _i32(index, B, accept_len, "accept_len"), W,
                              _i32(index, B, new_prefix_lens, "new_prefix_lens"), status,
                              _current_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SpecError(rc, "spec_kv4_compact")
    return new_prefix_lens


def tree_attn_kv4(q, kv_cache, prefix_lens, offsets, mask, max_prefix, status, o=None,
                  softmax_scale: float = 0.0, stream=None, parents=None, window: int = 0,
                  sinks: int = 0):
    """tree_attn over a 4-bit cache.  q [T, Hq, D] bf16 or fp32; with
    ``window`` > 0 a node sees only keys less than ``window`` positions behind
    it, and the first ``sinks`` positions; with ``mask=None`` the ancestor sets
    come from ``parents``."""
    lib = _lib or load()
    index, B, Hkv, S_cap, D = _kv4_cache(kv_cache)
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise TypeError("q must be bfloat16 or float32")
    shape = q.shape
    if len(shape) != 3 or shape[2] != D or q.get_device() != index or not q.is_contiguous():
        raise ValueError(f"q must be contiguous [T, Hq, {D}] on cuda:{index}")
    T, Hq, _ = shape
    mask_ptr = parents_ptr = None
    if mask is not None:
        mask_ptr = _i32(index, 4 * T, mask, "mask")
    elif parents is not None:
        parents_ptr = _i32(index, T, parents, "parents")
    else:
        raise ValueError("tree_attn_kv4 needs a mask or the parent array")
    if o is None:
        o = _new(stream, (T, Hq, D), (Hq * D, D, 1), q.dtype)
    elif o.dtype is not q.dtype or o.get_device() != index or o.shape != q.shape or not o.is_contiguous():
        raise ValueError("o must be like q")
    prefix, offsets, status = _per_request(index, B, prefix_lens, offsets, status, "prefix_lens")
    rc = lib.spec_tree_attn_kv4(q.data_ptr(), kv_cache.data_ptr(), o.data_ptr(), dt, B, T, Hq, Hkv, D, S_cap,
                                min(max_prefix, _INT_MAX), prefix, offsets, mask_ptr, parents_ptr, softmax_scale,
                                min(window, _INT_MAX), min(sinks, _INT_MAX), status,
                                _current_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SpecError(rc, "spec_tree_attn_kv4")
    return o


# ---------------------------------------------------------------- paged cache
class RopeTable(NamedTuple):
    """A rotation's frequencies: what rope and rope_write_paged take."""
    freqs: torch.Tensor       # [rotary_dim / 2] int64 (the bits of uint64), on the device
    scale: float              # of cosines and sines
    rotary_dim: int


_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
_I64 = torch.int64


def rope_table(rotary_dim, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=None, device="cuda"):
    """Frequencies of rotary positions over the first ``rotary_dim`` dims:
    base^(-2i / rotary_dim), for contexts ``factor`` times the ``original`` one
    scaled by "linear", "ntk", "yarn" or "bands" (spec_rope_table says how;
    ``high`` is 32 for "yarn" and 4 for "bands" unless given).  Computed on the
    host, once for a model."""
    kind = _ROPE_SCALINGS.get(scaling)
    if kind is None:
        raise ValueError(f"scaling is one of {', '.join(_ROPE_SCALINGS)}, not {scaling!r}")
    rotary_dim = int(rotary_dim)
    if not 2 <= rotary_dim <= 512:
        raise ValueError(f"rotary_dim is even and from 2 to 512, not {rotary_dim}")
    host = torch.zeros(rotary_dim // 2, dtype=_I64)
    scale = ctypes.c_float()
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    rc = load().spec_rope_table(rotary_dim, float(base), kind, float(factor), float(original), float(low), float(high),
                                host.data_ptr(), ctypes.byref(scale))
    if rc:
        raise SpecError(rc, "spec_rope_table")
    return RopeTable(host.to(device), scale.value, rotary_dim)


def _table(index, table):
    """(pointer, rotated dims, scale) of a rotation; None rotates nothing."""
    if table is None:
        return None, 0, 1.0
    freqs, scale, r = table
    if freqs.dtype is not _I64 or freqs.get_device() != index or 2 * freqs.numel() != r or not freqs.is_contiguous():
        raise ValueError(f"a rotation's frequencies are {r // 2} contiguous torch.int64 on cuda:{index}")
    return freqs.data_ptr(), r, scale


def _current(t, name):
    """The device index of a tensor, which is the current device's."""
    index = t.get_device()
    if index < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if index != _current_device():
        raise ValueError(f"{name} is on cuda:{index}, the current device is cuda:{_current_device()}")
    return index


def _pool(k_pages, v_pages, block_table, B):
    """Checks a paged cache; returns (device index, dtype code, pages, Hkv, page size, D, pages of a request)."""
    index, shape = _current(k_pages, "k_pages"), k_pages.shape
    dt = _DTYPES.get(k_pages.dtype)
    if dt is None or v_pages.dtype is not k_pages.dtype:
        raise TypeError("k_pages and v_pages must both be bfloat16 or float32")
    if (len(shape) != 4 or v_pages.shape != shape or v_pages.get_device() != index or not k_pages.is_contiguous()
            or not v_pages.is_contiguous()):
        raise ValueError(f"k_pages and v_pages must be contiguous [pages, Hkv, page_size, D] on cuda:{index}")
    if (block_table.dtype is not _I32 or block_table.get_device() != index or len(block_table.shape) != 2
            or block_table.shape[0] != B or not block_table.is_contiguous()):
        raise ValueError(f"block_table must be contiguous torch.int32 [{B}, max_pages] on cuda:{index}")
    if shape[0] > _INT_MAX or block_table.shape[1] > _INT_MAX:
        raise ValueError(f"a pool has at most {_INT_MAX} pages")
    return index, dt, shape[0], shape[1], shape[2], shape[3], block_table.shape[1]


def rope(x, table, start, offsets, status, depth=None, interleaved=False, out=None, stream=None):
    """Rotary positions on dense rows x [T, H, D] (bf16 or fp32; rows and heads
    at any stride): row t of request b at position start[b] + depth[t], or
    start[b] + t - offsets[b] without ``depth``.  ``out`` may be x (in place).
    Returns the rotated rows; a new tensor holds those of no request as they
    happen to be."""
    if _marshal is not None and out is None and stream is None:
        out = _marshal.rope(x, table, start, offsets, status, depth, interleaved)
        if out is not None:
            return out
    lib = _lib or load()
    index, dt = _current(x, "x"), _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError("x must be bfloat16 or float32")
    if len(x.shape) != 3:
        raise ValueError("x must be [T, H, D]")
    T, H, D = x.shape
    xs0, xs1 = _dense_rows(index, x, T, H, D, "x")
    freqs, r, scale = _table(index, table)
    if out is None:
        ys0, ys1 = H * D, D
        out = _new(stream, (T, H, D), (ys0, ys1, 1), x.dtype)
    else:
        if out.dtype is not x.dtype:
            raise TypeError(f"out must be {x.dtype}")
        ys0, ys1 = _dense_rows(index, out, T, H, D, "out")
    if depth is not None:
        depth = _i32(index, T, depth, "depth")
    B = status.numel()
    start, offsets, status = _per_request(index, B, start, offsets, status, "start")
    rc = lib.spec_rope(x.data_ptr(), out.data_ptr(), dt, B, T, H, D, xs0, xs1, ys0, ys1, freqs, r, scale,
                       1 if interleaved else 0, start, depth, offsets, status,
                       _current_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SpecError(rc, "spec_rope")
    return out


def rope_write_paged(q, k, v, k_pages, v_pages, block_table, prefix_lens, offsets, status, table=None, depth=None,
                     start=None, interleaved=False, q_out=None, stream=None):
    """New rows q [T, Hq, D] (or None), k, v [T, Hkv, D] (rows and heads at any
    stride) on their way into a paged cache: q rotated into a tensor of its
    own, k rotated and v copied to slots prefix_lens[b] and up of request b.
    Positions as in rope, from ``start`` or else prefix_lens on; without a
    ``table`` nothing is rotated.  Returns the rotated q."""
    if _marshal is not None and q_out is None and stream is None:
        q_out = _marshal.rope_write_paged(q, k, v, k_pages, v_pages, block_table, prefix_lens, offsets, status, table, depth,
                                          start, interleaved)
        if q_out is not None:
            return q_out
    lib = _lib or load()
    B = status.numel()
    index, dt, pages, Hkv, size, D, width = _pool(k_pages, v_pages, block_table, B)
    if k.dtype is not k_pages.dtype or v.dtype is not k_pages.dtype or (q is not None and q.dtype is not k.dtype):
        raise TypeError(f"rows must be of the cache's type, {k_pages.dtype}")
    T = k.shape[0]
    ks0, ks1 = _dense_rows(index, k, T, Hkv, D, "k")
    vs0, vs1 = _dense_rows(index, v, T, Hkv, D, "v")
    Hq = qs0 = qs1 = 0
    q_ptr = out_ptr = None
    if q is not None:
        if len(q.shape) != 3 or q.shape[1] < 1:
            raise ValueError(f"q must be [{T}, Hq, {D}]")
        Hq = q.shape[1]
        qs0, qs1 = _dense_rows(index, q, T, Hq, D, "q")
        if q_out is None:
            q_out = _new(stream, (T, Hq, D), (Hq * D, D, 1), q.dtype)
        elif (q_out.dtype is not q.dtype or q_out.get_device() != index or q_out.shape != q.shape
              or not q_out.is_contiguous()):
            raise ValueError("q_out must be contiguous, of q's shape and type")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    freqs, r, scale = _table(index, table)
    if depth is not None:
        depth = _i32(index, T, depth, "depth")
    if start is not None:
        start = _i32(index, B, start, "start")
    prefix, offsets, status = _per_request(index, B, prefix_lens, offsets, status, "prefix_lens")
    rc = lib.spec_rope_write_paged(q_ptr, out_ptr, k.data_ptr(), v.data_ptr(), dt, B, T, Hq, Hkv, D, qs0, qs1, ks0, ks1,
                                   vs0, vs1, freqs, r, scale, 1 if interleaved else 0, k_pages.data_ptr(),
                                   v_pages.data_ptr(), pages, size, block_table.data_ptr(), width, prefix, start,
                                   depth, offsets, status,
                                   _current_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SpecError(rc, "spec_rope_write_paged")
    return q_out


def tree_attn_paged(q, k_pages, v_pages, block_table, prefix_lens, offsets, mask, max_prefix, status, o=None,
                    softmax_scale: float = 0.0, stream=None, parents=None, causal=False):
    """Attention over a paged cache.  q [T, Hq, D] bf16 or fp32; trees by
    ``mask``, or by ``parents`` when it is None, as in tree_attn; with
    ``causal`` (mask and parents None) request b's rows are a run of any
    number of tokens behind its prefix, each seeing all before it.  Rows of
    ``o`` behind the last request stay as they were."""
    if _marshal is not None and o is None and stream is None:
        o = _marshal.tree_attn_paged(q, k_pages, v_pages, block_table, prefix_lens, offsets, mask, max_prefix, status,
                                     softmax_scale, parents, causal)
        if o is not None:
            return o
    lib = _lib or load()
    B = status.numel()
    index, dt, pages, Hkv, size, D, width = _pool(k_pages, v_pages, block_table, B)
    shape = q.shape
    if q.dtype is not k_pages.dtype:
        raise TypeError(f"q must be of the cache's type, {k_pages.dtype}")
    if len(shape) != 3 or shape[2] != D or q.get_device() != index or not q.is_contiguous():
        raise ValueError(f"q must be contiguous [T, Hq, {D}] on cuda:{index}")
    T, Hq, _ = shape
    if T > _INT_MAX or Hq > _INT_MAX:
        raise ValueError(f"q may have {_INT_MAX} rows and heads")
    mask_ptr = parents_ptr = None
    if causal:
        if mask is not None or parents is not None:
            raise ValueError("a causal run takes neither mask nor parents")
    elif mask is not None:
        mask_ptr = _i32(index, 4 * T, mask, "mask")
    elif parents is not None:
        parents_ptr = _i32(index, T, parents, "parents")
    else:
        raise ValueError("tree_attn_paged needs a mask, the parent array or causal=True")
    if o is None:
        o = _new(stream, (T, Hq, D), (Hq * D, D, 1), q.dtype)
    elif o.dtype is not q.dtype or o.get_device() != index or o.shape != q.shape or not o.is_contiguous():
        raise ValueError("o must be like q")
    prefix, offsets, status = _per_request(index, B, prefix_lens, offsets, status, "prefix_lens")
    rc = lib.spec_tree_attn_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), o.data_ptr(), dt, B, T, Hq,
                                  Hkv, D, pages, size, block_table.data_ptr(), width, min(max_prefix, _INT_MAX), prefix,
                                  offsets, mask_ptr, parents_ptr, 1 if causal else 0, softmax_scale, status,
                                  _current_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SpecError(rc, "spec_tree_attn_paged")
    return o


def kv_compact_paged(k_pages, v_pages, block_table, prefix_lens, offsets, path_nodes, accept_len, status,
                     new_prefix_lens=None, stream=None):
    """kv_compact on a paged cache (in place).  Returns the new prefix lengths
    (device int32 [B])."""
    if _marshal is not None and new_prefix_lens is None and stream is None:
        new_prefix_lens = _marshal.kv_compact_paged(k_pages, v_pages, block_table, prefix_lens, offsets, path_nodes,
                                                    accept_len, status)
        if new_prefix_lens is not None:
            return new_prefix_lens
    lib = _lib or load()
    B = status.numel()
    index, dt, pages, Hkv, size, D, width = _pool(k_pages, v_pages, block_table, B)
    W = path_nodes.shape[-1]
    if new_prefix_lens is None:
        new_prefix_lens = _new(stream, (B,), (1,), _I32)
    prefix, offsets, status = _per_request(index, B, prefix_lens, offsets, status, "prefix_lens")
    rc = lib.spec_kv_compact_paged(k_pages.data_ptr(), v_pages.data_ptr(), dt, B, Hkv, D, pages, size,
                                   block_table.data_ptr(), width, prefix, offsets,
                                   _i32(index, B * W, path_nodes, "path_nodes"),
                                   _i32(index, B, accept_len, "accept_len"), W,
                                   _i32(index, B, new_prefix_lens, "new_prefix_lens"), status,
                                   _current_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SpecError(rc, "spec_kv_compact_paged")
    return new_prefix_lens


def tree_expand(draft_logits, parent_scores, node_ids, requests, width: int, temperature: float,
                seed: int, stream=None):
    """One level of draft-tree expansion.  Returns (child_tokens [F][width],
    child_scores [F][width], near_ties [F][width]) as device tensors."""
    lib = load()
    _dev(draft_logits, torch.float32, "draft_logits")
    _dev(parent_scores, torch.float32, "parent_scores")
    _dev(node_ids, torch.int32, "node_ids")
    _dev(requests, torch.int32, "requests")
    F, V = draft_logits.shape
    dev_ = draft_logits.device
    tok = torch.empty((F, width), dtype=torch.int32, device=dev_)
    sc = torch.empty((F, width), dtype=torch.float32, device=dev_)
    ties = torch.empty((F, width), dtype=torch.int32, device=dev_)
    _check(lib.spec_tree_expand(_ptr(draft_logits), _ptr(parent_scores), _ptr(node_ids), _ptr(requests),
                                F, V, width, float(temperature), int(seed) & (2**64 - 1), _ptr(tok),
                                _ptr(sc), _ptr(ties), _stream(stream)), "spec_tree_expand")
    return tok, sc, ties


def tree_prune(parents, tokens, scores, cand_offsets, keep: int, status, stream=None):
    """Prune candidate trees to `keep` nodes.  Returns dict(parents, tokens,
    kept, n_out) of device tensors ([B][keep] rows)."""
    lib = load()
    for t, name in ((parents, "parents"), (tokens, "tokens"), (cand_offsets, "cand_offsets"),
                    (status, "status")):
        _dev(t, torch.int32, name)
    _dev(scores, torch.float32, "scores")
    B = cand_offsets.numel() - 1
    dev_ = parents.device
    out = {k: torch.empty((B, keep), dtype=torch.int32, device=dev_) for k in ("parents", "tokens", "kept")}
    out["n_out"] = torch.empty(B, dtype=torch.int32, device=dev_)
    _check(lib.spec_tree_prune(_ptr(parents), _ptr(tokens), _ptr(scores), _ptr(cand_offsets), B, keep,
                               _ptr(out["parents"]), _ptr(out["tokens"]), _ptr(out["kept"]),
                               _ptr(out["n_out"]), _ptr(status), _stream(stream)), "spec_tree_prune")
    return out


def philox_uniforms(seed: int, counters, out=None, stream=None):
    """Step R: the uniform for each counter row (c0, c1, c2, c3) of the int64
    device tensor ``counters`` [n, 4].  Returns a float32 device tensor [n]."""
    lib = load()
    _dev(counters, torch.int64, "counters")
    if counters.dim() != 2 or counters.shape[1] != 4:
        raise ValueError("counters must be [n, 4]")
    n = counters.shape[0]
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=counters.device)
    _check(lib.spec_philox_uniforms(int(seed) & (2**64 - 1), _ptr(counters), n, _ptr(out),
                                    _stream(stream)), "spec_philox_uniforms")
    return out


def tree_merge(parents_a, tokens_a, offsets_a, parents_b, tokens_b, offsets_b, status,
               stream=None):
    """Merge two speculators' token trees per request.  Returns dict(parents,
    tokens, map_b [B][128], n_out [B]) of device tensors."""
    lib = load()
    for t, name in ((parents_a, "parents_a"), (tokens_a, "tokens_a"), (offsets_a, "offsets_a"),
                    (parents_b, "parents_b"), (tokens_b, "tokens_b"), (offsets_b, "offsets_b"),
                    (status, "status")):
        _dev(t, torch.int32, name)
    B = offsets_a.numel() - 1
    if offsets_b.numel() - 1 != B:
        raise ValueError("both trees need the same number of requests")
    dev_ = parents_a.device
    out = {k: torch.empty((B, MAX_TREE_NODES), dtype=torch.int32, device=dev_)
           for k in ("parents", "tokens", "map_b")}
    out["n_out"] = torch.empty(B, dtype=torch.int32, device=dev_)
    _check(lib.spec_tree_merge(_ptr(parents_a), _ptr(tokens_a), _ptr(offsets_a), _ptr(parents_b),
                               _ptr(tokens_b), _ptr(offsets_b), B, parents_a.numel(),
                               parents_b.numel(), _ptr(out["parents"]), _ptr(out["tokens"]),
                               _ptr(out["map_b"]), _ptr(out["n_out"]), _ptr(status),
                               _stream(stream)), "spec_tree_merge")
    return out
