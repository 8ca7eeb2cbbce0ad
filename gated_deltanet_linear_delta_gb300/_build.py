"""Build the CUDA library libgdn_gb300.so in-tree with nvcc for sm_103a.

Each .cu file is compiled to an object in parallel, then linked into one
shared library with the CUDA runtime linked statically, so the library needs
only the NVIDIA driver at run time. binding.cpp becomes the CPython module
``_calls`` beside it, linked against that library and torch; where torch cannot
be imported the library is built alone. The results live in ``_lib/`` next to
this file (git-ignored).
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB_NAME = "libgdn_gb300.so"
CALLS_NAME = "_calls.so"
BINDING = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return cand


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _hash(paths: list[str], *words: str) -> str:
    h = hashlib.sha256(" ".join(words).encode())
    for p in paths:
        h.update(os.path.basename(p).encode())
        with open(p, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def _files(*dirs: str) -> list[str]:
    return [p for d in dirs for p in (os.path.join(d, f) for f in sorted(os.listdir(d))) if os.path.isfile(p)]


def _fingerprint() -> str:
    """Of all that the library is made from."""
    return _hash([p for p in _files(CSRC, INCLUDE) if p != BINDING], *ARCH, *NVCC_FLAGS)


def _torch_flags():
    """Compiler and linker flags of a CPython module that takes torch tensors; None without torch."""
    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    return ([f"-I{inc}", f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
             f"-I{sysconfig.get_paths()['include']}", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"],
            [f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"])


def _binding_fingerprint():
    """Of all that the module is made from; None without torch."""
    flags = _torch_flags()
    if flags is None:
        return None
    import torch
    return _hash([BINDING, *_files(INCLUDE)], torch.__version__, sysconfig.get_python_version(), *flags[0], *flags[1])


def lib_path() -> str:
    return os.path.join(OUT_DIR, LIB_NAME)


def calls_path() -> str:
    return os.path.join(OUT_DIR, CALLS_NAME)


def _fresh(stamp: str, built: str, fp: str) -> bool:
    if not (os.path.exists(built) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        return f.read().strip() == fp


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _link(cmd: list[str], to: str, stamp: str, fp: str, what: str) -> None:
    tmp = to + f".{os.getpid()}.tmp"
    _run([*cmd[:1], "-shared", "-o", tmp, *cmd[1:]], what)
    os.replace(tmp, to)
    with open(stamp, "w") as f:
        f.write(fp)


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile every .cu under csrc/ and link libgdn_gb300.so, and with torch the module for its tensors. Returns the
    library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    stamp, calls_stamp = os.path.join(OUT_DIR, "build.stamp"), os.path.join(OUT_DIR, "calls.stamp")
    fp, calls_fp = _fingerprint(), _binding_fingerprint()
    library = force or not _fresh(stamp, lib_path(), fp)
    calls = calls_fp is not None and (force or not _fresh(calls_stamp, calls_path(), calls_fp))
    cxx = shutil.which("g++") or "c++"

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        out = _run([nvcc(), *ARCH, *NVCC_FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", "-c", src, "-o", obj],
                   f"nvcc failed on {os.path.basename(src)}")
        if verbose and out.strip():
            print(out)
        return obj

    def compile_binding():
        obj = os.path.join(OUT_DIR, "binding.o")
        _run([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-I{INCLUDE}", *_torch_flags()[0], "-c", BINDING,
              "-o", obj], "g++ failed on binding.cpp")
        return obj

    srcs = sources() if library else []
    with cf.ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(compile_binding) if calls else None
        objs = list(ex.map(compile_one, srcs))
        binding_obj = binding.result() if calls else None
    if library:
        _link([nvcc(), *ARCH, "-cudart", "static", "-Xlinker", f"-soname={LIB_NAME}", *objs], lib_path(), stamp, fp,
              "link failed")
    if calls:
        _link([cxx, binding_obj, f"-L{OUT_DIR}", f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN", *_torch_flags()[1]], calls_path(),
              calls_stamp, calls_fp, "link of the binding failed")
    return lib_path()


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
