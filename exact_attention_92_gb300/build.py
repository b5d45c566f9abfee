"""Build libfa.so (the sm_103a CUDA library) in-tree with nvcc.

Each .cu file compiles to an object under ``_build/`` in parallel; the
objects link into ``exact_attention_92_gb300/libfa.so`` with the CUDA runtime
linked statically, so the library needs no libcudart at run time and loads on
a machine without a GPU driver (the tensor-map encoder is fetched from the
driver at first use).
"""

from __future__ import annotations

import concurrent.futures
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfa.so")
CALL_SOURCE = os.path.join(CSRC, "kv4_call.cpp")
CALL = os.path.join(PKG, "_kv4_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
PACKED_CALL_SOURCE = os.path.join(CSRC, "packed_call.cpp")
PACKED_CALL = os.path.join(PKG, "_packed_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_fwd256.cu", "fa_bwd.cu", "fa_bwd_pair.cu", "fa_bwd256.cu", "fa_noalloc.cu",
           "fa_kv4.cu", "fa_kv4_move.cu", "fa_kv4_fwd.cu", "fa_rope.cu", "fa_packed.cu", "fa_packed_fwd.cu",
           "fa_packed_bwd.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libfa.so")
    return cand


def _flags(extra=()):
    return ["-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
            "-I", INCLUDE, "-I", CSRC, *extra]


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "fa.h"), __file__]
    return max(os.path.getmtime(f) for f in files)


# Kernels that read tensor memory with tcgen05.ld: the destination registers
# of such a load are only valid after tcgen05.wait::ld, so a register spill
# between the two would store garbage.  The build refuses any spill in them.
NO_SPILL_KERNELS = ("fa_fwd_kernel", "fa_packed_fwd_kernel", "fa_fwd256_kernel", "fa_bwd_dkdv_kernel", "fa_bwd_dkdv_pair_kernel",
                    "fa_bwd_dq_kernel", "fa_bwd256_kv_kernel", "fa_bwd256_dq_kernel")


# Kernels that move registers between warpgroups with setmaxnreg, and the
# per-thread count they must be launched with.  The split's shares are
# static_asserted against this count in the source; if ptxas gave the entry
# fewer registers, the warpgroup that asks for more would wait forever.
REG_SPLIT_KERNELS = {"fa_fwd_kernel": 168, "fa_bwd_dkdv_kernel": 168, "fa_bwd_dkdv_pair_kernel": 168,
                     "fa_bwd_dq_kernel": 168, "fa_packed_fwd_kernel": 168}


def check_spills(ptxas_log: str) -> None:
    entry = None
    for line in ptxas_log.splitlines():
        m = re.search(r"Compiling entry function '([^']+)'", line)
        if m:
            entry = m.group(1)
            continue
        m = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", line)
        if m and entry and any(k in entry for k in NO_SPILL_KERNELS):
            if int(m.group(1)) or int(m.group(2)):
                raise RuntimeError(f"register spills in {entry}: {line.strip()}")
        m = re.search(r"Used (\d+) registers", line)
        if m and entry:
            for k, regs in REG_SPLIT_KERNELS.items():
                if k in entry and int(m.group(1)) != regs:
                    raise RuntimeError(f"{entry} starts with {m.group(1)} registers, its register split needs {regs}")


def _call_key(torch_dir: str) -> str:
    """What the native caller is compiled against: it holds the layout of
    torch's and CPython's objects."""
    import importlib.metadata

    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    st = os.stat(os.path.join(torch_dir, "lib", "libtorch_python.so"))
    return "\n".join([version, torch_dir, f"{st.st_size} {st.st_mtime_ns}", sys.version, sysconfig.get_paths()["include"]])


def build_call(force: bool = False) -> str | None:
    """Compile the native caller of the 4-bit cache's entry points (CALL)."""
    return _build_caller(CALL_SOURCE, CALL, "the 4-bit cache's calls", force)


def build_packed_call(force: bool = False) -> str | None:
    """Compile the native caller of rotary positions and packed sequences (PACKED_CALL)."""
    return _build_caller(PACKED_CALL_SOURCE, PACKED_CALL, "the calls on packed sequences", force)


def _build_caller(source: str, target: str, what: str, force: bool) -> str | None:
    """Compile a native caller (against torch's and Python's headers: again when
    those are other ones); None where torch with CUDA is not installed, and,
    with a warning, where it does not compile.  It holds no device code: without
    it the binding makes the same calls through ctypes."""
    import importlib.util

    spec = importlib.util.find_spec("torch")  # found, not imported
    if spec is None or not spec.submodule_search_locations:
        return None
    torch_dir = list(spec.submodule_search_locations)[0]
    inc, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    if not all(os.path.exists(os.path.join(lib, f)) for f in ("libc10_cuda.so", "libtorch_python.so")):
        return None
    key, key_file = _call_key(torch_dir), target + ".key"
    if not force and os.path.exists(target) and os.path.exists(key_file) and os.path.getmtime(target) >= max(
            os.path.getmtime(source), os.path.getmtime(os.path.join(INCLUDE, "fa.h")), os.path.getmtime(__file__)):
        with open(key_file, encoding="utf-8") as fh:
            if fh.read() == key:
                return target
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    tmp = target + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-I", INCLUDE, "-I",
           sysconfig.get_paths()["include"], source, "-o", tmp, "-L", lib, f"-Wl,-rpath,{lib}",
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        said = r.stdout + r.stderr
    except OSError as e:
        r, said = None, str(e)
    if r is None or r.returncode != 0:
        if os.path.exists(target):
            os.remove(target)  # of an older source, or against other headers
        warnings.warn(f"{what} go through ctypes: {cxx} failed on {source}:\n{said}")
        return None
    os.replace(tmp, target)
    with open(key_file, "w", encoding="utf-8") as fh:
        fh.write(key)
    return target


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link libfa.so if any source is newer than it, and the native
    callers (build_call, build_packed_call); return libfa.so's path."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=2) as ex:
        calls = [ex.submit(build_call, force), ex.submit(build_packed_call, force)]
        path = _build_lib(force, verbose, ptxas_verbose)
        for call in calls:
            call.result()
    return path


def _build_lib(force: bool, verbose: bool, ptxas_verbose: bool) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps() and not ptxas_verbose:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *_flags(extra), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    for _, log in results:
        check_spills(log)
    if verbose or ptxas_verbose:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of libfa.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas-v" in sys.argv))
