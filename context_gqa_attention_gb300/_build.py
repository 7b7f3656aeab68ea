"""In-tree build for sm_103a: libcpattn.so (nvcc, one object per source, parallel) and the Python
binding of its serving calls (the host compiler, against the torch that is installed)."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libcpattn.so")
BINDING = os.path.join(OUT_DIR, "cpattn_binding.so")
BUILT_FOR = os.path.join(OUT_DIR, "cpattn_binding.txt")  # the torch and Python that BINDING was built against
SOURCES = ["api.cu", "prefill_simt.cu", "prefill_tc.cu", "decode.cu", "noalloc.cu",
           "cache.cu", "decode_mod.cu", "decode_q4.cu", "prefill_mod.cu", "beam.cu", "cross.cu", "cross_few.cu", "cross_f32.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + ["binding.cpp"]]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "cpattn.h"))
    files.append(os.path.abspath(__file__))
    return files


def binding_target() -> str:
    """What a binding that fits this process was built against."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def binding_built_for() -> str:
    """What the binding on disk was built against ('' if there is none)."""
    if not (os.path.exists(BINDING) and os.path.exists(BUILT_FOR)):
        return ""
    with open(BUILT_FOR) as f:
        return f.read()


def up_to_date() -> bool:
    if not os.path.exists(LIB) or binding_built_for() != binding_target():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu for sm_103a and link libcpattn.so, and the binding, next to this file."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cxx = os.environ.get("CXX") or "g++"
    binding_obj = os.path.join(OUT_DIR, "binding.o")

    def compile_binding():
        cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE]
        for d in (sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
                  os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")):
            cmd += ["-isystem", d]
        r = subprocess.run([*cmd, "-c", os.path.join(CSRC, "binding.cpp"), "-o", binding_obj], capture_output=True,
                           text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cxx} failed on binding.cpp:\n{r.stderr}")

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        for obj, log in ex.map(compile_one, SOURCES):
            objs.append(obj)
            if verbose and log:
                print(log)
        binding.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if os.path.exists(BUILT_FOR):  # (written again once the binding it describes is in place)
        os.remove(BUILT_FOR)
    tmp = BINDING + ".tmp"
    cmd = [cxx, "-shared", "-o", tmp, binding_obj, "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", OUT_DIR, "-lcpattn", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BUILT_FOR, "w") as f:
        f.write(binding_target())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
