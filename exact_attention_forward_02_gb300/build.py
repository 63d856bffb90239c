"""Build libfa.so (the CUDA library behind the C ABI in include/*.h) in-tree.

Two CUDA translation units compiled at the same time, one -gencode (sm_103a), linked against
the static CUDA runtime; the driver entry point for TMA tensor maps is fetched at run time, so
no libcuda link. Beside it the tensor-level calls (_fa_torch.so), a host-only module over
libtorch: it is left out where there is no CUDA build of torch, which the library does not need.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SRCS = [os.path.join(CSRC, "fa_fwd.cu"), os.path.join(CSRC, "fa_decoder.cu")]
DEPS = SRCS + [os.path.join(CSRC, h) for h in ("sm103_ptx.cuh", "fa_bwd.cuh", "philox.cuh", "fa_fwd_kernel.cuh",
                                               "fa_rope.cuh", "fa_paged.cuh", "fa_host.h")] + [
    os.path.join(ROOT, "include", h) for h in ("fa_fwd.h", "fa_decoder.h")]
LIB = os.path.join(PKG, "libfa.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def compile_cmd(src: str, out: str, extra=()) -> list[str]:
    return [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-c", "-Xcompiler", "-fPIC",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC, *extra, src, "-o", out]


def link_cmd(objects, out: str) -> list[str]:
    return [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objects, "-o", out]


# The same library with device-side range checks of every stream-K workspace access
# (FA_DEBUG): an index outside the workspace's layout records FA_ERR_BOUNDS and the access
# is skipped. Used by the tests; the release library compiles the checks out.
DEBUG_LIB = os.path.join(PKG, "libfa_debug.so")
DEBUG_FLAGS = ("-DFA_DEBUG",)


# The tensor-level calls: a CPython module over libtorch's C++ API, host code only.
TORCH_SRC = os.path.join(CSRC, "fa_torch.cpp")
TORCH_DEPS = [TORCH_SRC] + [os.path.join(ROOT, "include", h) for h in ("fa_fwd.h", "fa_decoder.h")]
TORCH_LIB = os.path.join(PKG, "_fa_torch.so")


# the torch that the module on disk was compiled against
TORCH_STAMP = os.path.join(PKG, "_build", "torch_version")


def torch_root() -> str | None:
    """The folder of an installed torch that can be linked against for CUDA, or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    root = os.path.dirname(spec.origin)
    return root if os.path.exists(os.path.join(root, "lib", "libtorch_cuda.so")) else None


def torch_version(root: str) -> str:
    """What tells one build of torch from another (its version.py, and where it lies)."""
    path = os.path.join(root, "version.py")
    text = open(path).read() if os.path.exists(path) else ""
    return f"{root}\n{sys.version}\n{text}"


def _calls_stale(root: str) -> bool:
    if _stale(TORCH_LIB, TORCH_DEPS) or not os.path.exists(TORCH_STAMP):
        return True
    with open(TORCH_STAMP) as f:
        return f.read() != torch_version(root)


def torch_cmd(root: str, out: str) -> list[str]:
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    include = [os.path.join(ROOT, "include"), CSRC, os.path.join(root, "include"), cuda,
               sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *(x for i in include for x in ("-I", i)), TORCH_SRC,
            "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
            "-lc10_cuda", "-o", out]


def _stale(out: str, deps=None) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(out) < os.path.getmtime(d) for d in deps or DEPS)


def build(force: bool = False, verbose: bool = False, out: str = LIB, extra=()) -> str:
    return build_many([(out, extra)], force=force, verbose=verbose)[0]


def build_many(targets, force: bool = False, verbose: bool = False) -> list[str]:
    """Compile each (output, extra flags) target that is stale, all nvcc runs at once, and link it;
    with them the tensor-level calls, where torch can be linked."""
    procs, calls, torch = [], None, torch_root()
    if torch is None:
        sys.stderr.write(f"no CUDA build of torch: {os.path.basename(TORCH_LIB)} (the tensor-level calls) is not built\n")
    elif force or _calls_stale(torch):
        calls_tmp = TORCH_LIB + f".tmp{os.getpid()}"
        calls = subprocess.Popen(torch_cmd(torch, calls_tmp), stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
    for out, extra in targets:
        if force or _stale(out):
            objects = [f"{out}.{os.path.basename(src)}.tmp{os.getpid()}.o" for src in SRCS]
            flags = (*extra, "-Xptxas", "-v") if verbose else extra
            procs.append((out, objects, [
                subprocess.Popen(compile_cmd(src, obj, flags), stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
                for src, obj in zip(SRCS, objects)]))
    failed = []
    for out, objects, compiles in procs:
        said = [pr.communicate() for pr in compiles]
        ok = all(pr.returncode == 0 for pr in compiles)
        if ok:
            tmp = out + f".tmp{os.getpid()}"
            link = subprocess.run(link_cmd(objects, tmp), capture_output=True, text=True)
            said.append((link.stdout, link.stderr))
            ok = link.returncode == 0
        for obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
        if not ok:
            sys.stderr.write("".join(so + se for so, se in said))
            failed.append(os.path.basename(out))
            continue
        if verbose:
            sys.stderr.write("".join(se for _, se in said))
        os.replace(tmp, out)
    if calls is not None:
        so, se = calls.communicate()
        if calls.returncode == 0:
            os.replace(calls_tmp, TORCH_LIB)
            os.makedirs(os.path.dirname(TORCH_STAMP), exist_ok=True)
            with open(TORCH_STAMP, "w") as f:
                f.write(torch_version(torch))
        else:
            sys.stderr.write(so + se)
            failed.append(os.path.basename(TORCH_LIB))
    if failed:
        raise RuntimeError(f"the compiler failed building {', '.join(failed)}")
    return [out for out, _ in targets]


def build_all(force: bool = False) -> list[str]:
    """The release library and its range-checked twin."""
    return build_many([(LIB, ()), (DEBUG_LIB, DEBUG_FLAGS)], force=force)


if __name__ == "__main__":
    if "--all" in sys.argv:
        build_all(force="--force" in sys.argv)
    else:
        build(force="--force" in sys.argv, verbose="-v" in sys.argv)
