"""Builds the library: nvcc compiles each CUDA source for sm_103a, in parallel, and links
``libattn_gb300.so`` in the package directory (in-tree; git-ignored).  Beside it g++ compiles the quick
binding of the paged cache's calls against this machine's torch and Python, ``_binding.so`` (which those are, ``_build/_binding.stamp`` says); the library stands without it, and so
do the calls (paged.py), so that a machine where it cannot be built gets a warning."""
from __future__ import annotations

import os
import platform
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libattn_gb300.so")
BINDING = os.path.join(HERE, "_binding.so")
STAMP = os.path.join(BUILD, "_binding.stamp")
SOURCES = ["attn_api.cu", "fwd_f32.cu", "fwd_bf16_sm103.cu", "fwd_bf16_pair_sm103.cu", "decode.cu",
           "bwd.cu", "bwd_tc_sm103.cu", "qk_rope.cu", "paged_fwd.cu", "paged_rows.cu",
           "paged_rows_q8.cu", "paged_read_q8.cu", "paged_tc_sm103.cu", "paged_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v", "-I", os.path.join(HERE, "..", "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def binding_stamp() -> str:
    """What a quick binding is compiled against: one built for anything else is built anew, and not loaded."""
    import torch
    return " ".join(["torch", torch.__version__, "abi", str(int(torch._C._GLIBCXX_USE_CXX11_ABI)), str(sysconfig.get_config_var("SOABI")),
                     platform.machine()])


def binding_is_current() -> bool:
    """Whether there is a quick binding that was built for this torch and Python."""
    try:
        with open(STAMP) as f:
            return os.path.exists(BINDING) and f.read() == binding_stamp()
    except (ImportError, OSError):
        return False


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(HERE, "..", "include", "attn.h"))
    cc = nvcc()

    def compile_one(src):
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        if force or _stale(o, [s, *headers]):
            r = subprocess.run([cc, *ARCH, *FLAGS, "-c", s, "-o", o], capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
            log = os.path.join(BUILD, src + ".ptxas.txt")
            with open(log, "w") as f:
                f.write(r.stderr)
        return o

    def compile_binding():
        s = os.path.join(CSRC, "binding.cpp")
        if force or _stale(BINDING, [s, headers[-1]]) or not binding_is_current():
            for old in (STAMP, BINDING):
                if os.path.exists(old):
                    os.remove(old)  # an old one's parameter blocks may not be the library's
            import torch
            t = os.path.dirname(torch.__file__)
            tmp = BINDING + f".tmp{os.getpid()}"
            r = subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
                                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                                "-I", sysconfig.get_paths()["include"], "-I", os.path.join(t, "include"),
                                "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"), s, "-o", tmp,
                                "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-ldl"],
                               capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, BINDING)
            with open(STAMP, "w") as f:
                f.write(binding_stamp())

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    try:
        binding.result()
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the quick binding of the paged cache's calls was not built: {e}", RuntimeWarning)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
