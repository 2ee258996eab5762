"""Builds the CUDA library libmoe_gb300.so in-tree for sm_103a with nvcc.

Every translation unit is compiled in parallel to an object file, then linked into a
shared library next to this file (``_lib/libmoe_gb300.so``); the CPython marshalling of
``csrc/binding.c`` becomes ``_lib/_binding.<this interpreter's suffix>`` (gcc, Python's headers).
Either is rebuilt only when it is missing or one of its sources or headers is newer.
"""
import concurrent.futures as cf
import glob
import importlib.machinery
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libmoe_gb300.so")
BINDING_SRC = os.path.join(CSRC, "binding.c")
BINDING = os.path.join(OUT_DIR, "_binding" + importlib.machinery.EXTENSION_SUFFIXES[0])
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def python_include():
    return sysconfig.get_paths()["include"]


def stale():
    """The outputs that have to be built: LIB, BINDING, both or none."""
    headers = glob.glob(os.path.join(INCLUDE, "*.h"))
    deps = {LIB: sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + headers,
            BINDING: [BINDING_SRC] + headers}
    return {out for out, src in deps.items()
            if not os.path.exists(out) or any(os.path.getmtime(d) > os.path.getmtime(out) for d in src)}


def build(force: bool = False, verbose: bool = False) -> str:
    todo = {LIB, BINDING} if force else stale()
    if not todo:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc() if LIB in todo else None

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    def compile_binding():
        tmp = BINDING + ".tmp"
        cmd = ["gcc", "-O2", "-shared", "-fPIC", "-I" + python_include(), "-I" + INCLUDE, BINDING_SRC, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"gcc failed for {BINDING_SRC} (it needs Python.h):\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BINDING)

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding = ex.submit(compile_binding) if BINDING in todo else None
        if LIB in todo:
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + ".tmp"
            r = subprocess.run([cc] + ARCH + ["-shared", "-o", tmp] + objs, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        if binding:  # after the library: its calls work without the binding
            binding.result()
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
