"""Builds libsmoe.so in-tree from csrc/*.cu for sm_103a with nvcc.

Each translation unit is compiled in its own nvcc process (in parallel),
then linked into one shared library with the CUDA runtime linked
statically, so loading the library needs no GPU and no libcudart.
Two modules, _binding.so and _binding_f8.so (csrc/binding.c and binding_f8.c,
gcc, linked to libsmoe.so next to them), marshal the arguments of the calls that
small batches make; without Python's headers they are left out, and the package
makes those calls by ctypes.
Set SMOE_PTXAS_VERBOSE=1 to print register and shared-memory use, and
SMOE_NVCC_EXTRA to pass extra nvcc flags (e.g. -D tuning macros).
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsmoe.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_F8 = os.path.join(PKG, "_binding_f8.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.c")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _python_headers():
    """The folder of Python.h, or None."""
    d = sysconfig.get_paths()["include"]
    return d if os.path.exists(os.path.join(d, "Python.h")) else None


def up_to_date() -> bool:
    made = [LIB] + ([BINDING, BINDING_F8] if _python_headers() else [])
    if not all(os.path.exists(m) for m in made):
        return False
    t = min(os.path.getmtime(m) for m in made)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if os.environ.get("SMOE_PTXAS_VERBOSE") == "1":
        flags += ["-Xptxas", "-v"]
    flags += os.environ.get("SMOE_NVCC_EXTRA", "").split()  # extra compile flags (tuning builds)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose or os.environ.get("SMOE_PTXAS_VERBOSE") == "1":
            print(r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    headers = _python_headers()
    if headers is None:
        return LIB
    for made, source in ((BINDING, "binding.c"), (BINDING_F8, "binding_f8.c")):
        tmp = made + ".tmp"
        cmd = ["gcc", "-O2", "-shared", "-fPIC", "-I", INCLUDE, "-I", headers,
               os.path.join(CSRC, source), "-o", tmp, "-L", PKG, "-l:libsmoe.so", "-Wl,-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"gcc failed on {source}:\n{r.stderr}")
        os.replace(tmp, made)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
