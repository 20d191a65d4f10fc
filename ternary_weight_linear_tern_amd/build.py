"""Build libtern.so (the C-ABI HIP library) in-tree with hipcc for gfx950.

Usage: python -m ternary_weight_linear_tern_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libtern.so")
SOURCES = ["tern_kernels.hip", "tern_panel.hip", "tern_group.hip", "tern_optim.hip", "tern_noalloc.hip",
           "tern_recur.hip", "tern_q4.hip", "tern_ortho.hip", "tern_norm.hip", "tern_logprob.hip", "tern_distill.hip",
           "tern_api.cpp", "tern_layer.cpp", "tern_plan.cpp"]
ARCH = "gfx950"

# Packed FP32 VALU forms are turned off for all device code.
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    raise RuntimeError("hipcc not found")


def _run(cmd: list, cwd: str | None = None) -> str:
    """Run a compiler command; returns what it says on stderr, raises where it fails."""
    r = subprocess.run(cmd, capture_output=True, text=True, cwd=cwd)
    # hipcc's host pass does not know the device-only feature flag; drop that note
    noise = "'-packed-fp32-ops' is not a recognized feature for this target (ignoring feature)"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        sys.stderr.write(err + "\n")
        raise RuntimeError(f"hipcc failed ({r.returncode}): {' '.join(cmd)}")
    return err


def build(out: str = LIB, verbose: bool = False, save_temps_dir: str | None = None) -> str:
    """Compile every source, several at a time, and link the library."""
    common = [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC"]
    if save_temps_dir:
        common += ["-save-temps=obj"]
    jobs = max(1, min(int(os.environ.get("MAX_JOBS") or 8), os.cpu_count() or 1, len(SOURCES)))
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(jobs) as pool:
        objs = [os.path.join(save_temps_dir or tmp, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        cmds = [[*common, "-I", os.path.join(ROOT, "include"), *DEVICE_FLAGS, "-c", os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objs)]
        errs = list(pool.map(lambda c: _run(c, save_temps_dir), cmds))
        errs.append(_run([*common, "-shared", *objs, "-o", out + ".tmp"], save_temps_dir))
    if verbose and "".join(errs).strip():
        sys.stderr.write("\n".join(e for e in errs if e.strip()) + "\n")
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
