"""Builds the CUDA library in-tree with nvcc for sm_103a (the translation units in parallel)."""
from __future__ import annotations

import glob
import os
import subprocess
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")                  # the latent-cache verify call
CSRC_SERVING = os.path.join(PKG, "csrc_serving")  # grouped heads and the cache operators
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libmla_verify_attn.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC"]
_lock = threading.Lock()


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def units() -> list[str]:
    return sorted(f for d in (CSRC, CSRC_SERVING) for f in glob.glob(os.path.join(d, "*.cu")))


def sources() -> list[str]:
    return units() + sorted(f for d in (CSRC, CSRC_SERVING, INCLUDE) for e in ("*.cuh", "*.h")
                            for f in glob.glob(os.path.join(d, e)))


def is_stale(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc*/*.cu and link them into _build/libmla_verify_attn.so."""
    with _lock:
        if not force and not is_stale():
            return LIB_PATH
        os.makedirs(OUT_DIR, exist_ok=True)
        tag = ".%d.tmp" % os.getpid()
        include = [f for d in (INCLUDE, CSRC, CSRC_SERVING) for f in ("-I", d)]
        objs, jobs = [], []
        for src in units():
            obj = os.path.join(OUT_DIR, os.path.basename(src) + tag + ".o")
            cmd = [nvcc(), *NVCC_FLAGS, *include, "-c", "-o", obj, src]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            objs.append(obj)
            jobs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True)))
        try:
            said = [(cmd, p.communicate()[1], p.returncode) for cmd, p in jobs]
            for cmd, err, rc in said:
                _check(cmd, rc, err)
                if verbose:
                    print(err)
            tmp = LIB_PATH + tag
            cmd = [nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            _check(cmd, r.returncode, r.stderr)
            os.replace(tmp, LIB_PATH)
        finally:
            for obj in objs:
                if os.path.exists(obj):
                    os.remove(obj)
        return LIB_PATH


def _check(cmd, rc, err) -> None:
    if rc != 0:
        raise RuntimeError("nvcc failed (%d):\n%s\n%s" % (rc, " ".join(cmd), err[-4000:]))
