"""Build ``libspec_tree.so`` in-tree with nvcc for sm_103a (GB300).

Each ``csrc/*.cu`` file is compiled in parallel to an object under ``_build/``
and linked into one shared library next to this file.  The CUDA runtime is
linked statically, so the library needs only the driver at run time.

``build(checked=True)`` makes the bounds-checked debug build instead
(``-DSPEC_CHECKED``, objects under ``_build/spec_tree_checked``, output
``libspec_tree_checked.so``); ``binding.load()`` opens it when the
environment sets ``SPEC_TREE_CHECKED=1``.

``csrc/marshal.cpp`` becomes the module ``_marshal`` beside them (g++, torch's
headers): the paged calls' checks and launches from C++, which only saves
host time.  Its file is named after what it was compiled against (torch, this
Python, its source and the C header), and only a file of the right name is
loaded.  Where there is none, ``binding.py`` does that work.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libspec_tree.so")
BUILD_DIR = os.path.join(os.path.dirname(HERE), "_build", "spec_tree")
OUT_CHECKED = os.path.join(HERE, "libspec_tree_checked.so")
BUILD_DIR_CHECKED = os.path.join(os.path.dirname(HERE), "_build", "spec_tree_checked")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


MARSHAL_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared"]


def _marshal_sources() -> list[str]:
    return [os.path.join(CSRC, "marshal.cpp"), os.path.join(os.path.dirname(HERE), "include", "spec_tree.h")]


def marshal_path() -> str:
    """The file of the module ``_marshal`` for the present torch, Python and sources, whose layouts and
    signatures are compiled into it."""
    import torch
    key = hashlib.sha256(repr((torch.__version__, torch.version.git_version, sys.version, sysconfig.get_config_var("SOABI"),
                               MARSHAL_FLAGS)).encode())
    for path in _marshal_sources():
        with open(path, "rb") as f:
            key.update(hashlib.sha256(f.read()).digest())
    return os.path.join(HERE, f"_marshal_{key.hexdigest()[:16]}.so")


def build_marshal(force: bool = False) -> bool:
    """Builds the module ``_marshal``; False (and a line on stderr) if that fails.  Modules of
    other versions are removed, also when it fails."""
    try:
        import torch
        out = marshal_path()
        for old in glob.glob(os.path.join(HERE, "_marshal*.so")):
            if force or old != out:
                os.unlink(old)
        if os.path.exists(out):
            return True
        root = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
        inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
        lib = os.path.join(root, "lib")
        tmp = out + f".tmp{os.getpid()}"
        cmd = [os.environ.get("CXX", "g++"), *MARSHAL_FLAGS, *(f"-I{i}" for i in inc), _marshal_sources()[0], "-o", tmp,
               f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr[-2000:])
        os.replace(tmp, out)
        return True
    except Exception as e:
        print(f"_marshal was not built (calls take longer on the host): {e}", file=sys.stderr)
        return False


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers() -> list[str]:
    inc = os.path.join(os.path.dirname(HERE), "include")
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(inc, f) for f in os.listdir(inc) if f.endswith(".h")]
    return hs


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    build_dir = BUILD_DIR_CHECKED if checked else BUILD_DIR
    out = OUT_CHECKED if checked else OUT
    flags = FLAGS + (["-DSPEC_CHECKED"] if checked else [])
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    srcs = sources()
    hdrs = _headers()
    objs = [os.path.join(build_dir, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src, obj):
        if force or _stale(obj, [src] + hdrs):
            cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose:
                print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        marshal = ex.submit(build_marshal, force)
        list(ex.map(lambda p: compile_one(*p), zip(srcs, objs)))
        marshal.result()
    if force or _stale(out, objs):
        tmp = out + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
