"""Builds libpka.so (the CUDA kernels + C ABI) in-tree for sm_103a.

Each translation unit under csrc/ is compiled by nvcc in parallel, then the
objects are linked into paged_kv_attention_07_gb300/_build/libpka.so. Where torch with CUDA
is installed, the calls with torch tensors (csrc/torch_calls.cpp) become a Python module beside it.
Nothing is installed outside the repository.

    python -m paged_kv_attention_07_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
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
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libpka.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "pka.h"))
    return files


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir():
    """The directory of the installed torch with CUDA, or None: libpka.so itself needs none."""
    spec = importlib.util.find_spec("torch")
    path = os.path.dirname(spec.origin) if spec and spec.origin else None
    return path if path and os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def _torch_version(torch_dir: str) -> str:
    with open(os.path.join(torch_dir, "version.py")) as f:
        return re.search(r"^__version__\b[^=]*=\s*['\"]([^'\"]+)", f.read(), re.MULTILINE).group(1)


def torch_calls_path(torch_version: str) -> str:
    """The module of calls with torch tensors for that torch (its C++ interface is the version's) and this Python."""
    return os.path.join(OUT_DIR, f"_pka_torch.{torch_version}.{sysconfig.get_config_var('SOABI')}.so")


def _compile_torch_calls(torch_dir: str) -> str:
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    include = [INCLUDE, os.path.join(torch_dir, "include"), sysconfig.get_paths()["include"],
               os.path.join(cuda, "include")]
    obj = os.path.join(OUT_DIR, "torch_calls.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *[x for i in include for x in ("-I", i)], "-c",
           os.path.join(CSRC, "torch_calls.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_calls.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_torch_calls(obj: str, torch_dir: str, target: str) -> None:
    lib = os.path.join(torch_dir, "lib")
    tmp = f"{target}.{os.getpid()}.tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-l:libpka.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, target)


def _build_lib(verbose: bool, extra_flags) -> None:
    nvcc = _nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = f"{LIB}.{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile csrc/*.cu and link libpka.so, and the module of calls with torch tensors where torch is
    installed; what is up to date stays. Returns the library path."""
    deps = _deps() + [os.path.abspath(__file__)]
    torch_dir = _torch_dir()
    lib = force or _stale(LIB, deps)
    target = torch_calls_path(_torch_version(torch_dir)) if torch_dir else None
    calls = target is not None and (lib or _stale(target, [*deps, LIB]))
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        torch_obj = ex.submit(_compile_torch_calls, torch_dir) if calls else None
        if lib:
            _build_lib(verbose, extra_flags)
        if calls:
            _link_torch_calls(torch_obj.result(), torch_dir, target)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    verbose = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force=force, verbose=verbose or bool(extra), extra_flags=extra))
