"""In-tree build of libkvp.so (nvcc, sm_103a only) and of _kvp_calls.so, the
binding of its short calls (g++, against the installed torch, if there is one).

Each translation unit is compiled in parallel to an object under ``_build/``
and linked into ``_lib/``; an object is rebuilt when it is older than its source
or any header, that of _kvp_calls.so also when torch or Python is another.  No
cmake, no ninja.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libkvp.so")
CALLS_PATH = os.path.join(LIB_DIR, "_kvp_calls.so")
CALLS_KEY_PATH = os.path.join(LIB_DIR, "_kvp_calls.key")
CALLS_SOURCE = "kvp_calls.cpp"

SOURCES = [
    "kvp_api.cu",
    "kvp_append.cu",
    "kvp_decode_simt.cu",
    "kvp_decode_mma.cu",
    "kvp_decode_int8.cu",
    "kvp_decode_fp8.cu",
    "kvp_decode_fp8_umma.cu",
    "kvp_decode_int4.cu",
    "kvp_reduce.cu",
    "kvp_rope_append.cu",
    "kvp_tables.cu",
    "kvp_norm.cu",
    "kvp_matmul_fp8.cu",
    "kvp_matmul_fp8_pair.cu",
    "kvp_prefill.cu",
    "kvp_block_manager.cpp",
    "kvp_noalloc.cu",
    "kvp_selftest.cu",
]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O3",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def _cuda_home() -> str:
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _nvcc() -> str:
    cand = os.path.join(_cuda_home(), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None else None


def calls_key() -> str:
    """What _kvp_calls.so is built for: it holds the layouts of one torch's C++ types
    and one Python's."""
    torch_dir, torch = _torch_dir(), ""
    if torch_dir is not None:
        with open(os.path.join(torch_dir, "version.py")) as f:
            torch = f.read()
    return f"{sysconfig.get_config_var('SOABI')}\n{torch_dir}\n{torch}"


def calls_key_built() -> str | None:
    """calls_key() of the _kvp_calls.so that is there."""
    if not os.path.exists(CALLS_KEY_PATH):
        return None
    with open(CALLS_KEY_PATH) as f:
        return f.read()


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    hs += glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, ptxas_verbose: bool) -> tuple[str, str]:
    s = os.path.join(CSRC, src)
    o = os.path.join(BUILD_DIR, src + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", s, "-o", o]
    if src == CALLS_SOURCE:
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-I{INCLUDE}",
               f"-I{_torch_dir()}/include", f"-I{_cuda_home()}/include",
               f"-I{sysconfig.get_paths()['include']}", "-c", s, "-o", o]
    if ptxas_verbose and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
    return o, r.stderr


def _link(path: str, objs: list[str], cmd: list[str], anew: bool) -> None:
    if not anew and os.path.exists(path) and \
            os.path.getmtime(path) >= max(os.path.getmtime(o) for o in objs):
        return
    tmp = path + f".tmp{os.getpid()}"
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile (incrementally) and link libkvp.so, which needs nvcc alone, and
    _kvp_calls.so, where torch is installed; returns the former's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    hdr = _headers_mtime()
    torch_dir = _torch_dir()

    def obj(src):
        return os.path.join(BUILD_DIR, src + ".o")

    def stale(src):
        return force or ptxas_verbose or not os.path.exists(obj(src)) or \
            os.path.getmtime(obj(src)) < max(os.path.getmtime(os.path.join(CSRC, src)), hdr)

    key = calls_key()
    todo = [src for src in SOURCES if stale(src)]
    if torch_dir and (stale(CALLS_SOURCE) or calls_key_built() != key):
        todo.insert(0, CALLS_SOURCE)
        if os.path.exists(CALLS_KEY_PATH):
            os.remove(CALLS_KEY_PATH)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(todo), os.cpu_count() or 4))) as ex:
        jobs = {src: ex.submit(_compile, src, ptxas_verbose) for src in todo}
    calls = jobs.pop(CALLS_SOURCE, None)
    logs = [job.result()[1] for job in jobs.values()]
    objs = [obj(src) for src in SOURCES]
    _link(LIB_PATH, objs, [_nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-ldl"],
          force or bool(jobs))
    if calls is not None:
        logs.append(calls.result()[1])
    if torch_dir:
        lib = os.path.join(torch_dir, "lib")
        _link(CALLS_PATH, [obj(CALLS_SOURCE)],
              ["g++", "-shared", obj(CALLS_SOURCE), f"-L{LIB_DIR}", "-lkvp", f"-L{lib}",
               "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
               f"-Wl,-rpath,{lib}"], force or calls is not None)
        if calls_key_built() != key:
            tmp = CALLS_KEY_PATH + f".tmp{os.getpid()}"
            with open(tmp, "w") as f:
                f.write(key)
            os.replace(tmp, CALLS_KEY_PATH)
    if verbose or ptxas_verbose:
        for log in logs:
            if log.strip():
                print(log)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB_PATH)
