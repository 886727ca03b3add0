"""Build libinkling_rel_attn.so in-tree with nvcc for sm_100a, and the Python module
``_serving`` (csrc/serving_ext.cpp) with the host compiler against PyTorch.

Usage: ``python -m learned_relative_gqa_b200.build [--verbose]``.
The library is written next to this file; nothing is installed elsewhere.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libinkling_rel_attn.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
# the same library, with every shared / global index of the attention's forward and backward kernels
# checked (-DINKLING_BOUNDS_CHECK), for tests; the serving kernels hold no such checks
BOUNDS_CHECK_LIB_PATH = os.path.join(HERE, "libinkling_rel_attn_boundscheck.so")
# the serving calls on PyTorch tensors; it takes the library's entry points when that is loaded
EXT_SOURCE = os.path.join(CSRC, "serving_ext.cpp")
EXT_PATH = os.path.join(HERE, "_serving.so")
SOURCES = ["host.cu", "prep_kernels.cu", "fwd.cu", "bwd.cu", "l2clip.cu", "paged_cache.cu", "decode.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def stale(path: str = LIB_PATH) -> bool:
    """True when the library at `path` is missing or older than a source or header."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return any(os.path.getmtime(d) > t for d in deps)


def ext_unavailable() -> str:
    """Why the Python module cannot be built on this machine; empty where it can."""
    try:
        import torch  # noqa: F401
    except ImportError as e:
        return f"PyTorch cannot be imported ({e})"
    return "" if shutil.which("g++") else "there is no g++"


def ext_target() -> str:
    """What the Python module is built for: this interpreter and this PyTorch."""
    import sysconfig

    import torch
    return f"{sysconfig.get_config_var('SOABI')}, torch {torch.__version__}"


def ext_stale() -> bool:
    """True when the Python module is missing, older than a source, or built for another interpreter or PyTorch."""
    if stale(EXT_PATH):
        return True
    with open(EXT_PATH, "rb") as f:
        return f"serving module for {ext_target()}\0".encode() not in f.read()


def ext_command(out_path: str) -> list:
    """The host compiler's command line for the Python module."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda", "include")
    include = [INCLUDE, sysconfig.get_paths()["include"], cuda]
    torch_include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include")]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             f'-DINKLING_BUILT_FOR="{ext_target()}"', EXT_SOURCE, "-o", out_path]
            + [f"-I{d}" for d in include] + [a for d in torch_include for a in ("-isystem", d)]
            + [f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])


def build(force: bool = False, verbose: bool = False, out_path: str = LIB_PATH, defines: tuple = ()) -> str:
    """Compile the library and, with it, the Python module. ``defines`` / ``out_path`` build diagnostic
    variants of the library (for example ``INKLING_TRACE``) next to, not over, the product one.

    The library needs neither PyTorch nor the module: it is built without them too, and the serving
    calls of ``binding`` then say that the module is missing."""
    product = out_path == LIB_PATH and not defines
    due = force or not product or stale(LIB_PATH)
    why = ext_unavailable() if product else ""
    if why and due:
        print(f"{os.path.basename(EXT_PATH)} is not built: {why}", file=sys.stderr)
    module = product and not why and (due or ext_stale())
    procs, objs = [], []
    if due:
        build_dir = os.path.join(ROOT, "_build", "-".join(defines) or "default")
        os.makedirs(build_dir, exist_ok=True)
        common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", CSRC, "-I", INCLUDE,
                  "--expt-relaxed-constexpr"]
        if verbose:
            common += ["-Xptxas", "-v"]
        common += [f"-D{d}" for d in defines]
        for src in SOURCES:  # translation units compile side by side
            obj = os.path.join(build_dir, src.replace(".cu", ".o"))
            procs.append((subprocess.Popen(common + ["-c", os.path.join(CSRC, src), "-o", obj]), src))
            objs.append(obj)
    ext = subprocess.Popen(ext_command(EXT_PATH + ".tmp")) if module else None
    failed = [src for proc, src in procs if proc.wait() != 0]
    built = ext is not None and ext.wait() == 0
    if due and not failed:
        tmp = out_path + ".tmp"
        subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], check=True)
        if product and not built and os.path.exists(EXT_PATH):
            os.remove(EXT_PATH)  # an older module may not fit the new library
        os.replace(tmp, out_path)
    if built and not failed:  # nor a new one an older library
        os.replace(EXT_PATH + ".tmp", EXT_PATH)
    if ext is not None and not built:
        failed.append(os.path.basename(EXT_SOURCE))
    if failed:
        raise RuntimeError(f"the compiler failed on {', '.join(failed)}")
    return out_path


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
