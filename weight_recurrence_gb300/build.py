"""Builds liblinattn.so in-tree with nvcc for sm_103a (no cmake, no torch extension).

Each .cu translation unit compiles in parallel to an object under
``weight_recurrence_gb300/_build/``; one nvcc link makes
``weight_recurrence_gb300/lib/liblinattn.so`` with the CUDA runtime linked
statically, so the library depends on nothing but the driver.  The checked
variant (``--checked``) compiles the same sources with ``-DLA_CHECKED`` into
``_build_checked/`` and ``lib/liblinattn_checked.so``.  ``csrc/la_torch.cpp``,
the Python binding of part of the calls, compiles with g++ against the installed
PyTorch's headers into ``lib/_la_torch.so`` (it finds the library at run time);
without PyTorch the library is built alone, and another PyTorch than the binding
was made for makes it anew.

    python -m weight_recurrence_gb300.build [--force] [--verbose] [--checked]
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]
# release: the product library; checked: the same sources with -DLA_CHECKED,
# whose kernels test their computed indices against the buffers' extents and
# record LA_ERR_BOUNDS instead of making an access out of range
VARIANTS = {
    "release": ("_build", "liblinattn.so", []),
    "checked": ("_build_checked", "liblinattn_checked.so", ["-DLA_CHECKED"]),
}
BUILD = os.path.join(PKG, VARIANTS["release"][0])
LIB = os.path.join(LIBDIR, VARIANTS["release"][1])
LIB_CHECKED = os.path.join(LIBDIR, VARIANTS["checked"][1])
BINDING_SRC = os.path.join(CSRC, "la_torch.cpp")
BINDING = os.path.join(LIBDIR, "_la_torch.so")


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblinattn.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    inc = os.path.join(os.path.dirname(PKG), "include")
    hs += [os.path.join(inc, f) for f in os.listdir(inc) if f.endswith(".h")]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir():
    """Folder of the installed PyTorch (located, not imported), or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def torch_identity():
    """What the binding depends on besides its source: PyTorch's place and version and
    the interpreter's; None without PyTorch."""
    torch = _torch_dir()
    if torch is None:
        return None
    try:
        with open(os.path.join(torch, "version.py")) as f:
            version = f.read()
    except OSError:
        version = ""
    return "\n".join((sys.version, torch, version))


def binding_command(out: str):
    """g++ command line that makes the binding."""
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", *("-I" + i for i in inc), BINDING_SRC, "-o", out,
            "-L" + os.path.join(torch, "lib"), "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ltorch_python", "-ldl"]


def _read(path: str):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def build_variants(variants=("release",), force: bool = False, verbose: bool = False, extra_flags=()):
    """Compile (incrementally) every translation unit of the given variants and the
    binding at once, in parallel, then link each library; returns the library paths."""
    os.makedirs(LIBDIR, exist_ok=True)
    cc = nvcc()
    hdrs = headers()
    plan, procs = [], []
    bound = None
    made_for = os.path.join(PKG, VARIANTS["release"][0], "la_torch.made_for")
    identity = torch_identity()
    if identity is not None and (force or _read(made_for) != identity or
                                 _stale(BINDING, [BINDING_SRC, os.path.join(os.path.dirname(PKG), "include", "la.h")])):
        bound = BINDING + ".tmp%d" % os.getpid()
        procs.append((BINDING_SRC, subprocess.Popen(binding_command(bound), stdout=subprocess.PIPE,
                                                    stderr=subprocess.STDOUT)))
    for name in variants:
        bdir, libname, vflags = VARIANTS[name]
        bdir = os.path.join(PKG, bdir)
        os.makedirs(bdir, exist_ok=True)
        objs, started = [], 0
        for src in sources():
            obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
            objs.append(obj)
            if force or _stale(obj, [src] + hdrs):
                cmd = [cc, *ARCH, *NVCC_FLAGS, *vflags, *extra_flags, "-c", src, "-o", obj]
                if verbose:
                    print(" ".join(cmd), flush=True)
                procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
                started += 1
        plan.append((os.path.join(LIBDIR, libname), objs, started))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or verbose:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if bound and BINDING_SRC not in failed:
        os.replace(bound, BINDING)
        os.makedirs(os.path.dirname(made_for), exist_ok=True)
        with open(made_for, "w") as f:
            f.write(identity)
    if set(failed) - {BINDING_SRC}:
        raise RuntimeError("compilation failed for: " + ", ".join(failed))
    for lib, objs, started in plan:
        if force or started or _stale(lib, objs):
            tmp = lib + ".tmp%d" % os.getpid()
            cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.check_call(cmd)
            os.replace(tmp, lib)
    if failed:   # the libraries are there, the binding is not
        raise RuntimeError("compilation failed for: " + ", ".join(failed))
    return [lib for lib, _, _ in plan]


def build(force: bool = False, verbose: bool = False, extra_flags=(), checked: bool = False) -> str:
    """Compile (incrementally) and link one variant; returns the library path."""
    return build_variants(("checked" if checked else "release",), force, verbose, extra_flags)[0]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--checked", action="store_true", help="also build liblinattn_checked.so")
    a = ap.parse_args()
    names = ("release", "checked") if a.checked else ("release",)
    for path in build_variants(names, force=a.force, verbose=a.verbose):
        print(path)
