"""Build the HIP library ``libtsc.so`` in-tree for gfx950 with hipcc: the sampler's translation
unit (``csrc/``) and those of the operators around it (``csrc_ops/``), compiled side by side.

``python -m top_support_capture_amd.build`` (or ``build()``) always recompiles. The library is
placed next to this file, where the Python binding loads it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", "tsc_api.hip"),
           os.path.join(HERE, "csrc_ops", "ops_api.hip"),
           os.path.join(HERE, "csrc_ops", "logprob_api.hip"),
           os.path.join(HERE, "csrc_ops", "clip_api.hip")]
LIB = os.path.join(HERE, "libtsc.so")
ARCH = os.environ.get("TSC_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP library cannot be built")


def command(source: str, out: str) -> list:
    # Code object v5: loadable by the HIP runtime that PyTorch bundles as well as by /opt/rocm's.
    return [hipcc(), f"--offload-arch={ARCH}", "-mcode-object-version=5", "-O3", "-std=c++17",
            "-fPIC", "-c",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
            "-I", os.path.join(HERE, "csrc_ops"), "-o", out, source]


def _run(commands: list, verbose: bool) -> None:
    running = []
    for cmd in commands:
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append((cmd, subprocess.Popen(cmd)))
    failed = [cmd for cmd, p in running if p.wait() != 0]  # every compiler is waited for
    if failed:
        raise RuntimeError("failed: " + " ".join(failed[0]))


def build(verbose: bool = True) -> str:
    with tempfile.TemporaryDirectory(prefix="tsc_build_") as work:
        objects = [os.path.join(work, f"{i}.o") for i in range(len(SOURCES))]
        _run([command(s, o) for s, o in zip(SOURCES, objects)], verbose)
        tmp = LIB + ".tmp"
        _run([[hipcc(), f"--offload-arch={ARCH}", "-shared", "-o", tmp] + objects], verbose)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
