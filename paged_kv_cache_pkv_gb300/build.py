"""Build libpkv.so in-tree with nvcc for sm_103a (GB300).

Usage: python -m paged_kv_cache_pkv_gb300.build   (or call build()).
Each translation unit compiles in parallel; the shared library links the
CUDA runtime statically so it loads the same way under any PyTorch build.
_pkv_binding.so, the compiled argument checks of some calls, is host code
against this interpreter's and this PyTorch's headers.
"""

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
BINDING = os.path.join(HERE, "_pkv_binding.so")
SOURCES = ["pkv_api.cu", "pkv_write.cu", "pkv_decode.cu", "pkv_prefill.cu", "pkv_static.cu", "pkv_pool.cu",
           "pkv_rope.cu", "pkv_latent.cu", "pkv_latent_pair.cu", "pkv_evict.cu", "pkv_weigh.cu", "pkv_weigh_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _nvcc():
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else (shutil.which("nvcc") or "nvcc")


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_binding(force=False):
    """Compile the argument checks (csrc/pkv_binding.cpp) into BINDING."""
    import torch

    src = os.path.join(CSRC, "pkv_binding.cpp")
    include = os.path.join(os.path.dirname(HERE), "include")
    root = os.path.dirname(torch.__file__)
    if not (force or _stale(BINDING, [src, os.path.join(include, "pkv.h"), os.path.join(root, "version.py")])):
        return BINDING
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    dirs = [include, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    libs = os.path.join(root, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + d for d in dirs), src,
           "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           "-o", BINDING + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for pkv_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(verbose=False, force=False, extra_flags=(), lib_path=LIB, obj_dir=OUT_DIR):
    """Compile the sources into ``lib_path``; ``extra_flags`` (e.g. -D tuning
    macros) go to every nvcc call and need their own ``obj_dir``."""
    os.makedirs(obj_dir, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(os.path.dirname(HERE), "include", "pkv.h"))
    nvcc = _nvcc()

    def compile_one(src):
        s = os.path.join(CSRC, src)
        o = os.path.join(obj_dir, src + ".o")
        if force or _stale(o, [s] + headers):
            cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr, file=sys.stderr)
        return o

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, force) if lib_path == LIB else None
        objs = list(ex.map(compile_one, SOURCES))
        if binding:
            binding.result()
    if force or _stale(lib_path, objs):
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", *objs, "-o", lib_path + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(lib_path + ".tmp", lib_path)
    return lib_path


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv))
