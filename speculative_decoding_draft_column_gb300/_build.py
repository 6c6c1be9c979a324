"""Build ``libspecsel.so`` in-tree with nvcc for sm_103a (GB300)."""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SRCS = [os.path.join(CSRC, f) for f in ("specsel.cu", "paged.cu", "attention_tree.cu", "attention8.cu", "tree.cu")]
HDR = os.path.join(ROOT, "include", "specsel.h")
LIB = os.path.join(PKG, "libspecsel.so")

ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for c in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(c, "bin", "nvcc") if c else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecsel")
    return p


def command(out: str, srcs: list[str], extra: tuple[str, ...] = ()) -> list[str]:
    return [nvcc(), "-O3", "-std=c++17", ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
            "-cudart", "shared", "-I", os.path.join(ROOT, "include"), "-I", CSRC, *extra, "-o", out, *srcs]


def stale(out: str = LIB) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = [HDR, os.path.abspath(__file__)] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the sources in parallel, then link.  In a directory of its own,
    the library moved into place whole: builds at once do not mix, and a process
    that has the old library loaded keeps it."""
    if force or stale():
        with tempfile.TemporaryDirectory(prefix="_build", dir=os.path.dirname(LIB)) as tmp:
            objs = [os.path.join(tmp, os.path.splitext(os.path.basename(src))[0] + ".o") for src in SRCS]
            cmds = [command(o, [src], ("-c",)) for src, o in zip(SRCS, objs)]
            if verbose:
                print("\n".join(" ".join(c) for c in cmds), flush=True)
            procs = [subprocess.Popen(c) for c in cmds]
            codes = [p.wait() for p in procs]
            for cmd, rc in zip(cmds, codes):
                if rc != 0:
                    raise subprocess.CalledProcessError(rc, cmd)
            whole = os.path.join(tmp, os.path.basename(LIB))
            subprocess.run(command(whole, objs, ("-shared",)), check=True)
            os.replace(whole, LIB)
    return LIB
