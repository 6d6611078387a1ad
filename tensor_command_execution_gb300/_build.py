"""Build the CUDA executor library (libcmdexec.so) in-tree, and the module that hands torch tensors to its cache operators.

Each executor source compiles once per tier and op-set variant
(CMDX_TIER, CMDX_EXT; the tile executor also per view variant, CMDX_ND):
the per-tier interpreters are large, so this spreads them over parallel
compiler processes. With the host sources, all compile in parallel for
sm_103a only, then link into one shared library next to this file.
Float arithmetic is compiled with contraction off (-fmad=false) and without
fast-math, so denormals are kept and every add/sub/mul rounds once.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libcmdexec.so")
TORCH = importlib.util.find_spec("torch") is not None


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "unknown"


# (torch's C++ interface holds for one version of it)
TORCH_PATH = os.path.join(OUT_DIR, f"_cache_torch-{_torch_version() if TORCH else 'none'}.so")


# (source, the defines of each object built from it), longest compiles first
def _objs(tiers, nds=(None,)):
    out = []
    for t in tiers:
        for ext in (1, 0):
            for nd in nds:
                d = dict(CMDX_TIER=t)
                if nd is not None:
                    d["CMDX_ND"] = nd
                d["CMDX_EXT"] = ext
                out.append(d)
    return out


CU_SOURCES = [("exec_tile2d.cu", _objs((2,), (0, 1))), ("exec_generic.cu", _objs((2,))),
              ("exec_contig.cu", _objs((2,))), ("exec_contig.cu", [dict(CMDX_TIER=0, CMDX_EXT=1, CMDX_OCC4=1)]),
              ("exec_contig.cu", [dict(CMDX_TIER=1, CMDX_EXT=0, CMDX_HALF16=1)]),
              ("exec_tile2d.cu", _objs((1, 0), (0, 1))),
              ("exec_generic.cu", _objs((4, 3, 1, 0))), ("exec_contig.cu", _objs((4, 3, 1, 0))),
              ("static_scratch.cu", [{}]),
              ("cache_attend.cu", [{}]),
              ("cache_attend_mma.cu", [dict(CMDX_COPY=16), dict(CMDX_COPY=4)]),
              ("cache_attend_f32.cu", [dict(CMDX_COPY=16), dict(CMDX_COPY=4)]), ("cache_rope.cu", [{}]), ("cache_pages.cu", [{}])]
CPP_SOURCES = ["cmd_api.cpp", "cmd_yaml.cpp", "exec_host.cpp", "cache_api.cpp"]
TORCH_SOURCE = "cache_torch.cpp"
HEADERS = ["cmd_internal.h", "exec_common.cuh", "exec_pipe.cuh", "exec_tile2d.h", "interp_asm.cuh",
           "gen_interp.py", "cache_internal.h", "cache_common.cuh", "cache_attend.cuh",
           "cache_attend_ring.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def cuda_home() -> str:
    env = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if env and os.path.isdir(env):
        return env
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _sources():
    return ([os.path.join(CSRC, s) for s in sorted({c for c, _ in CU_SOURCES}) + CPP_SOURCES + [TORCH_SOURCE] + HEADERS]
            + [os.path.join(ROOT, "include", h) for h in ("cmd.h", "cmd_cache.h")] + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(s) <= t for s in _sources())


def _module_compile() -> str:
    """Compiles the module for torch tensors; returns its object file."""
    obj = os.path.join(OBJ_DIR, TORCH_SOURCE + ".o")
    torch_dir = _torch_dir()
    os.makedirs(OBJ_DIR, exist_ok=True)
    _step(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj,
           "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda_home(), "include"), "-I" + os.path.join(ROOT, "include")])
    return obj


def _module_link(obj: str) -> None:
    tmp = TORCH_PATH + f".tmp{os.getpid()}"
    _step(["g++", "-shared", "-o", tmp, obj, "-L" + os.path.join(_torch_dir(), "lib"), "-L" + OUT_DIR, "-ltorch_python",
           "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-l:libcmdexec.so", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, TORCH_PATH)


def _torch_dir() -> str:
    return list(importlib.util.find_spec("torch").submodule_search_locations)[0]


def _step(cmd: list) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def module_path() -> str:
    """The module that hands torch tensors to the cache operators, built first where it is missing or stale. The
    library does not depend on it: where it cannot be built (no headers of Python, a torch without CUDA), this is what
    raises."""
    build()
    if not TORCH:
        raise RuntimeError("the cache operators take torch tensors, and torch is not installed")
    sources = [os.path.join(CSRC, TORCH_SOURCE), os.path.join(ROOT, "include", "cmd.h"), os.path.join(ROOT, "include", "cmd_cache.h")]
    if not os.path.exists(TORCH_PATH) or os.path.getmtime(TORCH_PATH) < max(map(os.path.getmtime, sources)):
        try:
            _module_link(_module_compile())
        except Exception as e:
            raise RuntimeError(f"the cache operators' module for torch tensors could not be built: {e}") from e
    return TORCH_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libcmdexec.so unless it is newer than every source."""
    gen = os.path.join(CSRC, "gen_interp.py")
    inc_file = os.path.join(CSRC, "interp_asm.cuh")
    if not os.path.exists(inc_file) or os.path.getmtime(inc_file) < os.path.getmtime(gen):
        subprocess.run(["python3", gen], check=True, capture_output=True)
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    home = cuda_home()
    nvcc = os.path.join(home, "bin", "nvcc")
    inc = ["-I" + os.path.join(home, "include"), "-I" + os.path.join(ROOT, "include")]
    jobs = []
    for s, variants in CU_SOURCES:
        for defs in variants:
            stem = s + "".join(f".{k[5:].lower()}{v}" for k, v in defs.items())
            obj = os.path.join(OBJ_DIR, stem + ".o")
            log = os.path.join(OBJ_DIR, stem + ".ptxas.txt")
            cmd = ([nvcc] + ARCH + ["-O3", "-lineinfo", "-std=c++17", "-fmad=false", "-prec-div=true",
                                    "-prec-sqrt=true", "-ftz=false", "-Xptxas", "-v", "-Xcompiler", "-fPIC",
                                    "-c", os.path.join(CSRC, s), "-o", obj] + inc
                   + [f"-D{k}={v}" for k, v in defs.items()])
            jobs.append((cmd, obj, log))
    for s in CPP_SOURCES:
        obj = os.path.join(OBJ_DIR, s + ".o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra", "-Wno-unused-parameter",
               "-c", os.path.join(CSRC, s), "-o", obj] + inc
        jobs.append((cmd, obj, None))

    def run(job):
        cmd, obj, log = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        if log:
            with open(log, "w") as f:
                f.write(r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        module = ex.submit(_module_compile) if TORCH else None
        objs = list(ex.map(run, jobs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    link = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart_static", "-lrt", "-lpthread", "-ldl"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(link)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if os.path.exists(TORCH_PATH):
        os.remove(TORCH_PATH)  # (of an older build)
    if module:
        try:
            _module_link(module.result())
        except Exception as e:  # the first call that needs it tries again, and raises (module_path)
            if verbose:
                print(f"the module for torch tensors could not be built: {e}")
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
