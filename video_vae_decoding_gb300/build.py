"""Builds libwanvae.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each CUDA source is compiled in parallel to an object under ``_build/``,
then linked into ``libwanvae.so`` next to this file; the token operators'
marshalling in C++ becomes the Python module ``_tokens`` beside it, where it can
be made (the operators are marshalled in Python where not).  The CUDA runtime is
linked statically; the driver's tensor-map encoder is looked up at run time,
so the library loads on a machine without a GPU.
"""

from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libwanvae.so")
BINDING = os.path.join(HERE, "_tokens.so")
TAG = os.path.join(BUILD, "_tokens.tag")  # the Python and torch that BINDING was made for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libwanvae.so")


def sources() -> "list[str]":
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _csrc(*suffixes: str) -> "list[str]":
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(suffixes)]


def _headers() -> "list[str]":
    return [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")] + [os.path.abspath(__file__)]


def _newer(made: str, files: "list[str]") -> bool:
    return os.path.exists(made) and all(os.path.getmtime(f) <= os.path.getmtime(made) for f in files)


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    return list(spec.submodule_search_locations)[0]


def binding_tag() -> str:
    """The Python and the torch that the marshalling module is made for."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sys.implementation.cache_tag} torch {re.search(r'__version__ = .([^ ]+).$', f.read(), re.M).group(1)}"


def binding_fits() -> bool:
    """Whether the marshalling module beside this file was made for the Python and torch of this process."""
    try:
        with open(TAG) as f:
            return os.path.exists(BINDING) and f.read() == binding_tag()
    except (OSError, RuntimeError, AttributeError):
        return False


def library_up_to_date() -> bool:
    return _newer(LIB, _csrc(".cu", ".h", ".cuh") + _headers())


def binding_up_to_date() -> bool:
    return binding_fits() and _newer(BINDING, _csrc(".cpp") + _headers())


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _compile(nvcc: str, src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _link(nvcc: str, objs: "list[str]") -> None:
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _compile_binding() -> None:
    if os.path.exists(TAG):
        os.remove(TAG)  # one made of older sources is not used any more, whatever comes of this
    tmp, tag = BINDING + ".tmp", binding_tag()
    torch = _torch_dir()
    toolkit = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [INCLUDE, os.path.join(torch, "include"), sysconfig.get_paths()["include"],
                os.path.join(toolkit, "include")]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", *(f"-I{d}" for d in includes),
           os.path.join(CSRC, "token_binding.cpp"), "-o", tmp, "-L" + os.path.join(torch, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on token_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(TAG, "w") as f:
        f.write(tag)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles and links what is older than its sources; returns the library's path.

    The library does not depend on the marshalling module: where that cannot be
    made (it needs g++, Python's and torch's headers), this is said on stderr and
    the token operators are marshalled in Python."""
    library, binding = force or not library_up_to_date(), force or not binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc, srcs = (_nvcc(), sources()) if library else ("", [])
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        made = ex.submit(_compile_binding) if binding else None
        objs = list(ex.map(lambda src: _compile(nvcc, src, verbose), srcs))
        if library:
            _link(nvcc, objs)
        error = made.exception() if made else None
    if error is not None:
        sys.stderr.write(f"the token operators' marshalling in C++ was not built: {error}\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
