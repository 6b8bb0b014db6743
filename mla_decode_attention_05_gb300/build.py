"""Compile the CUDA library in-tree for sm_103a (GB300).

    python -m mla_decode_attention_05_gb300.build [--force] [--verbose-ptxas]

Each translation unit of csrc/ is compiled by its own nvcc process (in
parallel), then linked into _lib/libmla_decode.so with the CUDA runtime
linked statically, so the library loads on a machine without a GPU driver.
Beside it the host compiler makes _lib/fastcall-<hash>.so, the binding's short
way past the interpreter (csrc_host/), against the installed PyTorch.  The
binding does without it where it cannot be built: it only saves a call's time
on the host.
"""
from __future__ import annotations

import argparse
import contextlib
import glob
import hashlib
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(LIB_DIR, "obj")
SO = os.path.join(LIB_DIR, "libmla_decode.so")
FAST_SRC = os.path.join(HERE, "csrc_host", "fastcall.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _inputs():
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return srcs, deps


def up_to_date() -> bool:
    if not os.path.exists(SO):
        return False
    _, deps = _inputs()
    t = os.path.getmtime(SO)
    return all(os.path.getmtime(d) <= t for d in deps) and os.path.getmtime(__file__) <= t


def fast_path() -> str:
    """Where the short way is that was built from these sources for this
    interpreter and PyTorch.  The name holds what it depends on (it has
    accessors of PyTorch's tensors inlined, and calls the library through bare
    addresses), so one built for others is never found."""
    import sysconfig

    import torch
    h = hashlib.sha256()
    for part in (sysconfig.get_config_var("EXT_SUFFIX"), torch.__version__, torch.version.git_version):
        h.update(f"{part}\n".encode())
    for path in (FAST_SRC, os.path.join(INCLUDE, "mla_decode.h")):
        with open(path, "rb") as f:
            h.update(f.read())
    return os.path.join(LIB_DIR, f"fastcall-{h.hexdigest()[:16]}.so")


def _start_fast(force: bool):
    """Starts the host compiler on fastcall.cpp if it has to run -> (process,
    its output file, the file's name to be) or None.  Files of other sources,
    interpreters and PyTorches are removed first."""
    path = fast_path()
    for old in glob.glob(os.path.join(LIB_DIR, "fastcall*.so")):
        if force or old != path:
            with contextlib.suppress(FileNotFoundError):  # (another build removes them too)
                os.remove(old)
    if os.path.exists(path):
        return None
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), FAST_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), tmp, path
    except OSError as e:
        sys.stderr.write(f"fastcall.so not built: {e}\n")
        return None


def _finish_fast(started) -> None:
    if started is None:
        return
    pr, tmp, path = started
    text = pr.communicate()[0].decode(errors="replace")
    if pr.returncode == 0:
        os.replace(tmp, path)
    else:
        sys.stderr.write("fastcall.so not built (calls take longer on the host):\n" + text[-4000:])


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    fast = _start_fast(force)
    try:
        return _build_library(force, verbose_ptxas)
    finally:
        _finish_fast(fast)


def _build_library(force: bool, verbose_ptxas: bool) -> str:
    if not force and up_to_date():
        return SO
    nvcc = _nvcc()
    srcs, _ = _inputs()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]
    procs = []
    objs = []
    for s in srcs:
        o = os.path.join(OBJ_DIR, os.path.basename(s) + ".o")
        objs.append(o)
        procs.append((s, subprocess.Popen([nvcc, "-c", s, "-o", o] + flags,
                                          stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for s, pr in procs:
        out, _ = pr.communicate()
        text = out.decode(errors="replace")
        if pr.returncode != 0:
            failed.append((s, text))
        elif text.strip() and (verbose_ptxas or "warning" in text):
            sys.stderr.write(text)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError("nvcc failed:\n" + msg)
    tmp = SO + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static", "-ldl"])
    os.replace(tmp, SO)
    return SO


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
