"""Build libpagedkv.so in-tree for sm_103a with nvcc (translation units compiled in parallel), and the
binding's argument check (a small Python extension) with g++."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libpagedkv.so")
SOURCES = ["pkv_api.cu", "pkv_attn.cu", "pkv_attn_cols.cu", "pkv_attn_tc.cu", "pkv_cache_ops.cu",
           "pkv_rope.cu", "pkv_select.cu", "pkv_attn_blocks.cu", "pkv_verify.cu"]
HEADERS = ["pkv_device.cuh", "pkv_internal.h", "pkv_attn_common.cuh", "pkv_cols.cuh", "pkv_tcgen05.cuh",
           "pkv_cluster.cuh", "pkv_ops.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


ARGS_SOURCE = os.path.join(CSRC, "tensor_args.cpp")
ARGS_PATH = os.path.join(PKG, "tensor_args" + sysconfig.get_config_var("EXT_SUFFIX"))


def args_built_for(torch) -> str:
    """The interpreter and the torch whose layouts are compiled into the binding's argument check: it is used with no others."""
    return (f"python {sys.version.split()[0]} {sysconfig.get_config_var('EXT_SUFFIX')}, torch {torch.__version__} "
            f"{torch.version.git_version}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def start_tensor_args(force: bool = False):
    """Start compiling the binding's argument check if it is older than its source or was built for another Python or
    torch; None if there is nothing to do.  It needs the headers of both; without them the binding checks in Python."""
    python = sysconfig.get_paths()["include"]
    try:  # the library itself needs neither of them
        import torch
    except ImportError:
        torch = None
    stamp = ARGS_PATH + ".for"
    if not force and torch is not None and os.path.exists(ARGS_PATH) and os.path.exists(stamp) and open(stamp).read() == args_built_for(
            torch) and os.path.getmtime(ARGS_PATH) >= max(os.path.getmtime(f) for f in (ARGS_SOURCE, os.path.join(INCLUDE, "pkv.h"))):
        return None
    if torch is None or not shutil.which("g++") or not os.path.exists(os.path.join(python, "Python.h")):
        print("tensor_args is not built (no torch, no g++ or no Python.h): the binding checks its arguments in Python", file=sys.stderr)
        return None
    base = os.path.dirname(torch.__file__)
    tmp = ARGS_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBUILT_FOR="{args_built_for(torch)}"', "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"), "-I", python, "-I", INCLUDE, ARGS_SOURCE,
           "-o", tmp, "-L", os.path.join(base, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python", "-ldl"]
    return tmp, args_built_for(torch), subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def finish_tensor_args(started) -> None:
    if started is None:
        return
    tmp, built_for, proc = started
    text, _ = proc.communicate()
    if proc.returncode == 0:
        os.replace(tmp, ARGS_PATH)
        with open(ARGS_PATH + ".for", "w") as f:
            f.write(built_for)
    else:
        print("tensor_args is not built, the binding checks its arguments in Python:\n" + text.decode(errors="replace")[-2000:],
              file=sys.stderr)


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libpagedkv needs the CUDA toolkit to build")


def _stale(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "pkv.h"),
                                                                  os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
                  out: str | None = None, defines=(), build_dir: str | None = None) -> str:
    """Compile every .cu to an object in _build/, link libpagedkv.so next to this file.

    ``out``/``defines``/``build_dir`` build a variant elsewhere (e.g. the test build with
    -DPKV_TEST_HOOKS, or other pipeline depths via -DPKV_STAGES=...; a variant is rebuilt when any
    source is newer than it, so give each set of defines its own ``out`` and ``build_dir``); the
    default build is the in-tree library the package loads.
    """
    variant = out is not None
    out = out or LIB_PATH
    bdir = build_dir or BUILD_DIR
    fresh = not force and not _stale(out)
    nvcc = None if fresh else nvcc_path()
    started = None if variant else start_tensor_args(force)
    if fresh:
        finish_tensor_args(started)
        return out
    os.makedirs(bdir, exist_ok=True)
    common = [nvcc, "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", INCLUDE, "-I", CSRC, *[f"-D{d}" for d in defines]]
    if ptxas_info:
        common += ["-Xptxas", "-v"]
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(bdir, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    logs = []
    failed = []
    for src, p in procs:
        text, _ = p.communicate()
        logs.append(text.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    finish_tensor_args(started)
    log_text = "".join(logs)
    with open(os.path.join(bdir, "compile.log"), "w") as f:
        f.write(log_text)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}:\n{log_text}")
    tmp = out + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, out)
    if verbose:
        print(log_text, file=sys.stderr)
    return out


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
