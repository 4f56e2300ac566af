"""Builds libbeam_moe.so (HIP, gfx950) in-tree from csrc/, and _bind.so, the
native argument marshalling of the Python package's attention calls.

Every call compiles from scratch: each .hip file to an object under
_build/, then the shared libraries next to this file.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(HERE, "libbeam_moe.so")
BIND_PATH = os.path.join(HERE, "_bind.so")
SOURCES = ["beam_moe.hip", "route.hip", "permute.hip", "experts.hip", "combine_norm.hip", "pack.hip", "mx.hip",
           "beam_attn.hip", "attn_prep.hip", "attn_decode.hip"]

ARCH = "gfx950"
HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # keep the compiler from emitting packed fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE,
]


def hipcc() -> str:
    env = os.environ.get("HIPCC")
    if env:
        return env
    for cand in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC)")


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed: " + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def build(verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = hipcc()
    jobs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        jobs.append((obj, [cc, *HIP_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]))
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
        outs = list(ex.map(lambda j: _run(j[1]), jobs))
    if verbose:
        for o in outs:
            if o.strip():
                print(o)
    tmp = LIB_PATH + ".tmp"
    _run([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *[j[0] for j in jobs], "-o", tmp])
    os.replace(tmp, LIB_PATH)
    _build_bind(cc, extra_flags)
    return LIB_PATH


def _build_bind(cc: str, extra_flags) -> None:
    import torch   # its DLPack header; nothing of torch is linked
    tmp = BIND_PATH + ".tmp"
    _run([cc, *HIP_FLAGS, *extra_flags, "-I", os.path.join(os.path.dirname(torch.__file__), "include"),
          "-I", sysconfig.get_paths()["include"], "-shared", os.path.join(CSRC, "bind.hip"), "-o", tmp])
    os.replace(tmp, BIND_PATH)


if __name__ == "__main__":
    print(build(verbose=True))
