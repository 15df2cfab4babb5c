"""Build libdiffattn.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu file under csrc/ is compiled to an object in parallel, then linked
into differential_attention_fwd_gb300/libdiffattn.so.  Objects go to
_build/ at the repository root.  A rebuild happens only when a source or
header is newer than the library.

csrc/binding.cpp, the Python binding of the paged-cache operators, is compiled with
the host compiler against torch's headers into _binding.so beside the library,
which it calls; it fits that torch alone, whose version _build/binding.torch keeps.
Either is made again by itself, and an error of the binding leaves the library in
place: the C ABI needs nothing but nvcc.

build(variant="waitprof") makes a second library, libdiffattn_waitprof.so,
from the same sources compiled with -DDIFFATTN_WAIT_PROFILE: its forward
kernel also counts the cycles each warp role spends waiting on barriers
(diffattn_wait_profile reads them).  It is a measurement build only; the
product is libdiffattn.so.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdiffattn.so")
BINDING = os.path.join(PKG, "_binding.so")
VARIANTS = {
    None: (LIB, BUILD, []),
    "waitprof": (os.path.join(PKG, "libdiffattn_waitprof.so"), os.path.join(BUILD, "waitprof"),
                 ["-DDIFFATTN_WAIT_PROFILE"]),
}

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdiffattn.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _binding_command(obj: str):
    """(compile, link) commands of the binding, for the torch that is installed."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
                "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
                "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    link = [cxx, "-shared", obj, "-o", BINDING + ".tmp", "-L", PKG, "-l:libdiffattn.so", "-L", lib, "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _headers():
    return sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))) + _headers()


def _newer(lib: str, deps) -> bool:
    return os.path.exists(lib) and all(os.path.getmtime(p) <= os.path.getmtime(lib) for p in deps)


def up_to_date(lib: str = LIB) -> bool:
    return _newer(lib, _deps())


def torch_version():
    """The version of the torch that imports, or None."""
    try:
        import torch
    except ImportError:
        return None
    return str(torch.__version__)


def _stamp() -> str:
    return os.path.join(BUILD, "binding.torch")


def binding_torch():
    """The version of the torch that the binding was built for, or None where it is not known."""
    if not os.path.exists(_stamp()):
        return None
    with open(_stamp()) as f:
        return f.read()


def binding_up_to_date() -> bool:
    return (_newer(BINDING, [os.path.join(CSRC, "binding.cpp"), *_headers()]) and
            binding_torch() is not None and binding_torch() == torch_version())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          variant=None) -> str:
    """Compile and link what is not up to date; returns the library path.  The library needs nvcc
    alone, and is in place before the binding (which needs torch's headers) can fail."""
    lib, objdir, defines = VARIANTS[variant]
    with_lib = force or not up_to_date(lib)
    with_binding = variant is None and (force or not binding_up_to_date())
    if not with_lib and not with_binding:
        return lib
    cc = nvcc()
    os.makedirs(objdir, exist_ok=True)
    extra = (["-Xptxas", "-v"] if ptxas_info else []) + defines

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    def compile_binding():
        compile_, link = _binding_command(os.path.join(objdir, "binding.cpp.o"))
        _run(compile_, "the binding does not compile")
        return link

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        link_binding = ex.submit(compile_binding) if with_binding else None
        results = list(ex.map(compile_one, _sources())) if with_lib else []
    if verbose or ptxas_info:
        for obj, log in results:
            if log.strip():
                print(f"== {os.path.basename(obj)}\n{log}", file=sys.stderr)
    if with_lib:
        tmp = lib + ".tmp"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if with_binding:
        _run(link_binding.result(), "the binding does not link")
        os.replace(BINDING + ".tmp", BINDING)
        with open(_stamp(), "w") as f:
            f.write(torch_version() or "")
    return lib


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
