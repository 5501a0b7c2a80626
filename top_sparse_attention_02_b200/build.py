"""Build libtsa.so (the CUDA kernels and the C ABI) in-tree with nvcc for sm_100a.

Also builds libtsa_debug.so, a test-only variant of the same sources whose
bounded device waits give up after a few polls and which exports two knobs,
tsa_debug_skip_tile (the decode step's kernels) and tsa_debug_paged_skip_tile
(the paged ones), that leave a chosen tile's load out so that the waits on it
run out (the failure-detection tests).  The product library has neither.

What a build was made from is told by content, not by time: each object lies
beside the digest of its source, the headers and the flags, and a library holds
the digest of all of them, so that ensure() knows whether it has to be built."""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtsa.so")
BUILD_DIR = os.path.join(PKG, "_build")
DEBUG_LIB = os.path.join(PKG, "libtsa_debug.so")
DEBUG_BUILD_DIR = os.path.join(PKG, "_build_debug")
DEBUG_FLAGS = ["-DTSA_WAIT_SPINS=1024", "-DTSA_DEBUG_KNOBS"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _digest(files: list, debug: bool) -> str:
    h = hashlib.sha256(repr(ARCH + [f for f in FLAGS if not os.path.isabs(f)] + (DEBUG_FLAGS if debug else [])).encode())
    for f in files:
        with open(f, "rb") as fh:
            data = fh.read()
        h.update(f"{os.path.basename(f)} {len(data)}\n".encode())
        h.update(data)
    return h.hexdigest()


def _mark(debug: bool) -> str:
    return "tsa-sources:" + _digest(sources() + _headers(), debug)


def _is(path: str, digest: str) -> bool:
    try:
        with open(path) as f:
            return f.read() == digest
    except OSError:
        return False


def current(debug: bool = False) -> bool:
    """Whether the library is there and was built from the sources as they are."""
    try:
        with open(DEBUG_LIB if debug else LIB, "rb") as f:
            return _mark(debug).encode() in f.read()
    except OSError:
        return False


def ensure(debug: bool = False) -> str:
    """The library's path; built first unless it is current.  Without nvcc a library of other
    sources is an error."""
    if not current(debug):
        lib = DEBUG_LIB if debug else LIB
        try:
            _nvcc()
        except RuntimeError as e:
            raise RuntimeError(f"{lib} is missing or was not built from these sources, and cannot be built here: {e}") from None
        build(debug=debug)
    return DEBUG_LIB if debug else LIB


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile every csrc/*.cu to an object (in parallel), then link libtsa.so
    (debug: the same sources with DEBUG_FLAGS into libtsa_debug.so)."""
    nvcc = _nvcc()
    build_dir, lib, extra = (DEBUG_BUILD_DIR, DEBUG_LIB, DEBUG_FLAGS) if debug else (BUILD_DIR, LIB, [])
    os.makedirs(build_dir, exist_ok=True)
    headers = _headers()
    mark = _mark(debug)
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        objs.append(obj)
        digest = _digest([src] + headers, debug)
        if force or not os.path.exists(obj) or not _is(obj + ".id", digest):
            if os.path.exists(obj + ".id"):
                os.remove(obj + ".id")
            log = open(obj + ".log", "w")
            procs.append((src, subprocess.Popen([nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj],
                                                stdout=log, stderr=subprocess.STDOUT), obj, digest))
    failed = []
    for src, p, obj, digest in procs:
        if p.wait() != 0:
            failed.append((src, obj + ".log"))
        else:
            with open(obj + ".id", "w") as f:
                f.write(digest)
    if failed:
        msg = "\n".join(f"--- {s}\n" + open(l).read() for s, l in failed)
        raise RuntimeError("nvcc failed:\n" + msg)
    if verbose:
        for _, _, obj, _ in procs:
            sys.stdout.write(open(obj + ".log").read())
    if force or procs or not current(debug):
        ident = os.path.join(build_dir, "source_id.cu")
        with open(ident, "w") as f:
            f.write(f'extern "C" __attribute__((visibility("default"))) const char tsa_source_id[] = "{mark}";\n')
        tmp = lib + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, ident, *objs])
        os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
