"""Build libemusgemm (the CUDA library behind the C ABI) in-tree for sm_103a.

Each .cu file under csrc/ is compiled by nvcc in parallel and the objects are
linked into ``csrc/_build/libemusgemm.<machine>.so``.  The CUDA runtime is
linked statically; the driver's tensor-map encoder is looked up at run time,
so the library has no link-time dependency on libcuda.  The Python side of
emu_layers.h, a CPython extension, is compiled beside it by the host compiler
where torch is installed.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import platform
import shutil
import subprocess
import sysconfig
from importlib import metadata

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(CSRC, "_build")
LIB_NAME = f"libemusgemm.{platform.machine()}.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)

SOURCES = ["emu_sgemm.cu", "split.cu", "gemm_kblock.cu", "gemm_simt.cu", "noalloc.cu", "chooser.cu",
           "gated.cu", "gemm_few.cu", "lora.cu", "qk_norm.cu"]
HEADERS = ["emu_device.cuh", "emu_host.h", "emu_internal.h", "gated.cuh", "schedule.h"]


def _torch_version():
    """None where there is no torch: the C library needs none."""
    try:
        return metadata.version("torch")
    except metadata.PackageNotFoundError:
        pass
    try:
        import torch
    except ImportError:
        return None
    return torch.__version__


# the Python side of emu_layers.h: a CPython extension against torch's headers
# (None where torch is missing)
BIND_SOURCE = "layers_bind.cpp"
TORCH = _torch_version()
BIND_PATH = TORCH and os.path.join(BUILD_DIR, f"emu_layers_bind.{platform.machine()}.{TORCH}.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libemusgemm")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_command(out: str) -> list[str]:
    import torch
    at = os.path.dirname(torch.__file__)
    include = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(at, "include"),
               os.path.join(at, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *(f"-I{d}" for d in include),
            os.path.join(CSRC, BIND_SOURCE), "-o", out, f"-L{os.path.join(at, 'lib')}",
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, h) for h in ("emu_sgemm.h", "emu_layers.h")]
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", f".{platform.machine()}.o"))
        objs.append(o)
        if force or _stale(o, [s, *headers]):
            jobs.append([cc, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compilation failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return r

    cuda_jobs = len(jobs)
    bind_tmp = f"{BIND_PATH}.tmp{os.getpid()}"
    bind_stale = BIND_PATH is not None and (
        force or _stale(BIND_PATH, [os.path.join(CSRC, BIND_SOURCE), *headers[-2:], __file__]))
    if bind_stale:
        jobs.append(_bind_command(bind_tmp))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    if bind_stale:
        os.replace(bind_tmp, BIND_PATH)
    if cuda_jobs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        run([cc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
