"""Build libmsa.so, the sm_103a MSA library, in-tree with nvcc.

Each ``csrc/*.cu`` is compiled in parallel to an object under ``_build/`` and
the objects are linked into ``libmsa.so`` next to this file (CUDA runtime
linked statically, so the library needs only the driver at run time).
``csrc/binding.cpp`` becomes ``_msa_binding``, the Python module that checks
and marshals torch tensors for the serving-step calls; it finds ``libmsa.so``
beside itself.  Objects are rebuilt when their source or any header is newer, the
module's also for another torch or interpreter; what is linked, when an object is newer.
The library does not depend on the module: where that cannot be built (no Python
headers), ``libmsa.so`` is there all the same, and an older module is not.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmsa.so")
BINDING = os.path.join(HERE, "_msa_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")
    return cand


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, obj: str, extra) -> str:
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _compile_binding(src: str, obj: str, extra) -> str:
    """binding.cpp against torch's and this interpreter's headers."""
    import torch
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    at = os.path.join(os.path.dirname(torch.__file__), "include")
    inc = [at, os.path.join(at, "torch", "csrc", "api", "include"), sysconfig.get_path("include"),
           os.path.join(cuda, "include"), os.path.join(cuda, "targets", f"{os.uname().machine}-linux", "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DMSA_BUILT_FOR="{torch.__version__}"', "-I", INCLUDE,
           *[x for d in inc for x in ("-isystem", d)], "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(src)}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return ""


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libmsa.so", f"-L{libs}", "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def _binding_stamp() -> str:
    """What a built module depends on besides its source and headers."""
    import torch
    return f"torch {torch.__version__} cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} python {sys.version} {os.path.basename(BINDING)}"


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _older(target: str, *sources: str) -> bool:
    return not os.path.exists(target) or os.path.getmtime(target) < max(os.path.getmtime(s) for s in sources)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every CUDA source for sm_103a and link libmsa.so and the Python module; returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr = _headers_mtime()

    def due(src, obj):
        return force or _older(obj, src) or os.path.getmtime(obj) < hdr

    objs = [os.path.join(BUILD, os.path.splitext(os.path.basename(s))[0] + ".o") for s in srcs]
    jobs = [(_compile, s, o) for s, o in zip(srcs, objs) if due(s, o)]
    bind_src, bind_obj, stamp = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, "binding.o"), os.path.join(BUILD, "binding.stamp")
    bind_due = due(bind_src, bind_obj) or _read(stamp) != _binding_stamp()
    if bind_due:
        jobs.append((_compile_binding, bind_src, bind_obj))
    if bind_due or _older(BINDING, bind_obj):
        # one laid out by other headers must not meet the new library
        for old in glob.glob(os.path.join(os.path.dirname(BINDING), "_msa_binding*.so")):
            os.remove(old)
    failed = None
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = {ex.submit(f, s, o, list(extra_flags) + (["-Xptxas", "-v"] if verbose else [])): s
                    for f, s, o in jobs}
            for f in cf.as_completed(futs):
                try:
                    log = f.result()
                except RuntimeError as e:
                    if futs[f] != bind_src:
                        raise
                    failed = e                  # the library first
                    continue
                if verbose and log:
                    sys.stderr.write(log)
    if force or _older(LIB, *objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if failed is not None:
        raise failed
    if force or _older(BINDING, bind_obj):
        _link_binding(bind_obj)
    if bind_due:
        with open(stamp, "w") as f:
            f.write(_binding_stamp())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
