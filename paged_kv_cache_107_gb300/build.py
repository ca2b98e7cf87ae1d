"""Build the CUDA library in-tree: paged_kv_cache_107_gb300/lib/libpagedkv.so.

Every .cu file under csrc/ is compiled for sm_103a only (one -gencode), in parallel, then
linked into one shared library with a plain C ABI (include/pa.h). No torch headers are
involved; the CUDA runtime is linked statically. Beside it goes the Python module of
csrc/py_call.c, lib/_pa_call with the running interpreter's extension suffix, where a C compiler
and Python.h are there (the binding goes through ctypes without it).
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
CSRC = os.path.join(HERE, "csrc")
LIB_DIR = os.path.join(HERE, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libpagedkv.so")
CALL_SRC = os.path.join(CSRC, "py_call.c")
# (the suffix names the interpreter and the machine: a module of another one is not taken for it)
CALL_PATH = os.path.join(LIB_DIR, "_pa_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
OBJ_DIR = os.path.join(LIB_DIR, "obj")
GENCODE = "arch=compute_103a,code=sm_103a"


def _nvcc() -> str:
    cuda_home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH") or "/usr/local/cuda"
    cand = os.path.join(cuda_home, "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: set CUDA_HOME")
    return found


def _flags(extra=()):
    return ["-gencode", GENCODE, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
            "--expt-relaxed-constexpr", *extra]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + [os.path.join(os.path.dirname(HERE), "include", "pa.h")]


def _lib_up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def up_to_date() -> bool:
    return _lib_up_to_date() and (_call_up_to_date() or _call_tools() is None)


def _call_up_to_date() -> bool:
    if not os.path.exists(CALL_PATH):
        return False
    header = os.path.join(os.path.dirname(HERE), "include", "pa.h")
    t = os.path.getmtime(CALL_PATH)
    return all(os.path.getmtime(p) <= t for p in (CALL_SRC, header))


def _call_tools():
    """(C compiler, folder of Python.h), None where one is missing."""
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    include = sysconfig.get_paths()["include"]
    return (cc, include) if cc and os.path.exists(os.path.join(include, "Python.h")) else None


def build_call():
    """Compile csrc/py_call.c for the running interpreter. Returns the module's path, or None
    without a C compiler or Python.h."""
    tools = _call_tools()
    if tools is None:
        sys.stderr.write("csrc/py_call.c not compiled: no C compiler (CC) or no Python.h\n")
        return None
    cc, include = tools
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = CALL_PATH + f".tmp{os.getpid()}"
    cmd = [cc, "-O2", "-std=gnu11", "-shared", "-fPIC", "-I", include, CALL_SRC, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cc} failed for {CALL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL_PATH)
    return CALL_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=(), lib_path: str = None) -> str:
    """Compile csrc/*.cu for sm_103a and link lib/libpagedkv.so, and the Python module beside it,
    as far as they are not up to date. Returns the library's path.

    lib_path: build a separate library there instead (always rebuilt, objects beside it),
    for example a test build with extra preprocessor flags; the in-tree library is left
    alone."""
    if lib_path is not None:
        return _build_to(lib_path, lib_path + ".obj", verbose, extra_flags)
    if force or not _lib_up_to_date():
        _build_to(LIB_PATH, OBJ_DIR, verbose, extra_flags)
    if force or not _call_up_to_date():
        build_call()
    return LIB_PATH


def _build_to(lib_path: str, obj_dir: str, verbose: bool, extra_flags) -> str:
    os.makedirs(obj_dir, exist_ok=True)
    nvcc = _nvcc()
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, *_flags(extra_flags), "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = lib_path + f".tmp{os.getpid()}"
    cmd = [nvcc, "-gencode", GENCODE, "-shared", "-Xcompiler", "-fPIC", "-o", tmp,
           *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
