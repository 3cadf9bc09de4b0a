"""Builds libs2attn.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m sparse_attention_attn_b200.build          # build if sources changed
    python -m sparse_attention_attn_b200.build --force  # always rebuild
    python -m sparse_attention_attn_b200.build --debug  # libs2attn_debug.so: kernels with index checks

The library is plain CUDA C++ compiled by nvcc; it links only the CUDA runtime
(statically) and resolves cuTensorMapEncodeTiled through the runtime's driver
entry-point query, so it needs no libcuda at link time.

Beside it, _s2torch.so: a small CPython extension (g++, torch's headers) that
shortens the Python side of the smallest calls.  Where it cannot be built the
package works without it.
"""
from __future__ import annotations

import hashlib
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libs2attn.so")
LIB_DEBUG = os.path.join(PKG, "libs2attn_debug.so")
BINDING = os.path.join(PKG, "_s2torch.so")
BINDING_SOURCE = os.path.join(CSRC, "s2_torch.cpp")

SOURCES = ["s2attn.cu", "s2_fwd.cu", "s2_fwd64.cu", "s2_bwd.cu", "s2_bwd_fused.cu", "s2_rope.cu", "s2_segment.cu", "s2_nf4.cu", "s2_bwd_ds.cu", "s2_bwd_kv128.cu",
           "s2_qknorm.cu", "s2_cache.cu", "s2_cache_dec.cu", "s2_cache_tc.cu"]
HEADERS = ["s2_ptx.cuh", "s2_common.cuh", "s2_cache.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libs2attn.so")


def header_hash() -> str:
    """Name of the interface in include/s2attn.h; compiled into the library and
    into _s2torch.so, which calls the library by address."""
    with open(os.path.join(INCLUDE, "s2attn.h"), "rb") as fh:
        return "h" + hashlib.sha256(fh.read()).hexdigest()[:16]


def source_hash(debug: bool = False) -> str:
    h = hashlib.sha256()
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "s2attn.h")]
    for f in files:
        with open(f, "rb") as fh:
            h.update(os.path.basename(f).encode())
            h.update(fh.read())
    h.update(" ".join(ARCH).encode())
    h.update(__file__.encode())
    h.update(b"debug" if debug else b"release")
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile libs2attn.so (or, with debug, libs2attn_debug.so: the same
    sources with the kernels' index checks compiled in) unless an up-to-date
    build exists, and with it _s2torch.so.  Returns its path.  The sources
    compile in parallel."""
    if not debug:
        try:
            built = build_binding(force)
            why = "no compiler or headers for it"
        except (OSError, subprocess.CalledProcessError) as e:
            built, why = None, e
        if built is None:
            print(f"warning: _s2torch.so was not built ({why}); the Python path serves alone", file=sys.stderr)
    lib = LIB_DEBUG if debug else LIB
    stamp = lib + ".srchash"
    digest = source_hash(debug)
    if not force and os.path.exists(lib) and os.path.exists(stamp):
        with open(stamp) as fh:
            if fh.read().strip() == digest:
                return lib
    nvcc = nvcc_path()
    tmpdir = os.path.join(PKG, "_build_debug" if debug else "_build")
    os.makedirs(tmpdir, exist_ok=True)
    common = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                     "-I" + INCLUDE, "-I" + CSRC, "--expt-relaxed-constexpr", "-DS2ATTN_HEADER_HASH=" + header_hash()]
    if debug:
        common += ["-DS2ATTN_DEBUG_CHECKS"]
    if verbose:
        common += ["-Xptxas", "-v"]
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(tmpdir, src.replace(".cu", ".o"))
        procs.append((src, subprocess.Popen([nvcc] + common + ["-c", os.path.join(CSRC, src), "-o", obj])))
        objs.append(obj)
    failed = [src for src, p in procs if p.wait() != 0]
    if failed:
        raise RuntimeError(f"nvcc failed on {', '.join(failed)}")
    tmp_lib = lib + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp_lib] + objs
    subprocess.run(cmd, check=True)
    os.replace(tmp_lib, lib)
    with open(stamp, "w") as fh:
        fh.write(digest)
    return lib


BINDING_FLAGS = ["-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden"]


def _torch_home():
    """Torch's folder and its version (located and read, not imported); (None, None) without it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None, None
    home = os.path.dirname(spec.origin)
    try:
        with open(os.path.join(home, "version.py")) as fh:
            named = dict(re.findall(r"^(__version__|git_version)\b[^=]*= '([^']*)'", fh.read(), re.M))
    except OSError:
        return None, None
    return home, f"{named.get('__version__')} {named.get('git_version')}"


def binding_command(source: str, out: str, optimize: str = "-O2"):
    """The command that compiles a binding source; None where a compiler or headers are missing."""
    gxx, python_h = shutil.which("g++"), sysconfig.get_paths()["include"]
    home, version = _torch_home()
    if home is None or gxx is None:
        return None
    cuda_h = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")
    torch_h = os.path.join(home, "include")
    if not all(map(os.path.exists, (os.path.join(python_h, "Python.h"), os.path.join(torch_h, "ATen", "ATen.h"),
                                    os.path.join(cuda_h, "cuda_runtime.h")))):
        return None
    return [gxx, optimize, *BINDING_FLAGS, f'-DS2ATTN_HEADER_HASH="{header_hash()}"', f'-DS2TORCH_VERSION="{version}"',
            "-I" + INCLUDE, "-I" + python_h, "-I" + torch_h,
            "-I" + os.path.join(torch_h, "torch", "csrc", "api", "include"), "-I" + cuda_h, source,
            "-L" + os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
            "-o", out]


def build_binding(force: bool = False):
    """Compile _s2torch.so unless an up-to-date build exists.  Returns its
    path, or None where a compiler or headers are missing.  A build of other
    sources or for another torch is removed first: it would call the library by
    an old interface, or read torch's tensors by an old layout."""
    stamp, tmp = BINDING + ".srchash", BINDING + ".tmp"
    h = hashlib.sha256(f"{BINDING_FLAGS} {sys.version} {_torch_home()[1]} {header_hash()}".encode())
    with open(BINDING_SOURCE, "rb") as fh:
        h.update(fh.read())
    if not force and os.path.exists(BINDING) and os.path.exists(stamp):
        with open(stamp) as fh:
            if fh.read().strip() == h.hexdigest():
                return BINDING
    for old in (stamp, BINDING):
        if os.path.exists(old):
            os.remove(old)
    cmd = binding_command(BINDING_SOURCE, tmp)
    if cmd is None:
        return None
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(stamp, "w") as fh:
        fh.write(h.hexdigest())
    return BINDING


if __name__ == "__main__":
    path = build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv)
    print(path)
