"""Builds libcpattn.so in-tree (next to this file) with nvcc for sm_103a.

    python context_long_sequence_zigzag_gb300/build.py

Each translation unit is compiled in parallel into ``_build/`` and linked
into one shared library with the CUDA runtime linked statically, so the
library only needs the NVIDIA driver at run time.  Objects are rebuilt when a
source or header is newer.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import platform
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build", platform.machine())
LIB = os.path.join(PKG, "libcpattn.so")

SOURCES = [
    "cp_attn_host.cu",
    "simple_kernels.cu",
    "device_status.cu",
    "attn_fwd_sm103.cu",
    "attn_bwd_sm103.cu",
    "linear_attn.cu",
    "linear_attn_tc.cu",
    "key_weights_sm103.cu",
    "kv4_host.cu",
    "kv4_cache.cu",
    "kv4_attn.cu",
    "kv_host.cu",
    "rope.cu",
    "kv_attn.cu",
    "kv_pages.cu",
]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills,-v"]
# Registers a thread that kernels have to come out with: their warps hand them to one another, and the launcher refuses
# any other count (kLaunchRegs in kv_attn.cu).
REGISTERS = {"kv_attn_kernel": 128}


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    hs = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    hs += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs


def _stale(obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def check_registers(log: str) -> None:
    """Raises if the assembler's report names a kernel of REGISTERS with another count."""
    kernel = ""
    for line in log.splitlines():
        m = re.search(r"Compiling entry function '(\w+)'", line)
        if m:
            kernel = m.group(1)
        m = re.search(r"Used (\d+) registers", line)
        for name, want in REGISTERS.items():
            if m and name in kernel and int(m.group(1)) != want:
                raise RuntimeError(f"{kernel}: {m.group(1)} registers, {want} are needed")


def build(verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdrs = _headers()
    flags = FLAGS + list(extra_flags or [])
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if _stale(o, [s] + hdrs):
            jobs.append([nvcc, *ARCH, *flags, "-I", INCLUDE, "-I", CSRC, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for cmd, r in ex.map(run, jobs):
                if verbose or r.returncode != 0:
                    sys.stderr.write(r.stdout + r.stderr)
                if r.returncode != 0:
                    raise RuntimeError("nvcc failed: " + " ".join(cmd))
                try:
                    check_registers(r.stderr)
                except RuntimeError:
                    os.remove(cmd[-1])  # (or the next build would link it)
                    raise
    if jobs or _stale(LIB, objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-Xcompiler", "-fPIC", "-ldl"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("link failed: " + " ".join(cmd))
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
