"""Build the SDM C-ABI library (libsdm.so) in-tree for sm_100a with nvcc."""
from __future__ import annotations

import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsdm.so")
OBJ = os.path.join(HERE, "_build")  # one object per source, rebuilt when an input is newer
SOURCES = [os.path.join(CSRC, "sdm_api.cu"), os.path.join(CSRC, "ssm_api.cu")]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _inputs(source=None):
    """Files the library (or the object of one source) is built from: the source and what it
    includes from csrc and include, followed through the quoted includes."""
    todo = [source] if source else list(SOURCES)
    files = []
    while todo:
        f = todo.pop()
        if f in files:
            continue
        files.append(f)
        with open(f) as fh:
            for name in re.findall(r'^\s*#include "([^"]+)"', fh.read(), flags=re.M):
                for d in (os.path.dirname(f), os.path.join(ROOT, "include")):
                    if os.path.exists(os.path.join(d, name)):
                        todo.append(os.path.normpath(os.path.join(d, name)))
                        break
    return files


def _newer(target, files) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def _object(source) -> str:
    return os.path.join(OBJ, os.path.splitext(os.path.basename(source))[0] + ".o")


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile libsdm.so unless it is newer than every source.  Returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
             "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), *extra]
    jobs = []
    for src in SOURCES:  # the sources compile side by side
        obj = _object(src)
        if not force and _newer(obj, _inputs(src)):
            continue
        cmd = [NVCC, *flags, "-c", "-o", obj + f".tmp{os.getpid()}", src]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        jobs.append((obj, cmd, subprocess.Popen(cmd)))
    codes = [p.wait() for _, _, p in jobs]
    for (obj, cmd, _), rc in zip(jobs, codes):
        if rc != 0:
            raise subprocess.CalledProcessError(rc, cmd)
        os.replace(obj + f".tmp{os.getpid()}", obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                    "--cudart=static", "-Xcompiler", "-fPIC", "-o", tmp,
                    *[_object(s) for s in SOURCES]], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
