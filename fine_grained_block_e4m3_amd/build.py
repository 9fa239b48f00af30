"""Build libfp8gemm.so (HIP, gfx950 only) in-tree.

    python -m fine_grained_block_e4m3_amd.build [--asm]

The library is compiled ahead of time with hipcc; there is no runtime JIT.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp8gemm.so")
SOURCES = [os.path.join(CSRC, name) for name in ("fp8gemm_api.hip", "ffn_api.hip", "skinny_launch.hip", "routing_api.hip")]
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # packed FP32 VALU forms are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # FP32 division must be the correctly rounded IEEE operation (quantizers)
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-fast-math",
    # MFMA results in VGPRs: the promotion FMAs read them without v_accvgpr_read
    # "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall",
    f"-I{os.path.join(ROOT, 'include')}",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


def _run(cmd: list, verbose: bool, cwd: str | None = None) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True, cwd=cwd)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l and "(ignoring feature)" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)


def build(asm_dir: str | None = None, verbose: bool = False) -> str:
    """Compile every HIP source and link libfp8gemm.so.  Always recompiles;
    the sources are compiled side by side."""
    out = LIB
    work = tempfile.mkdtemp(prefix="fp8gemm_build")
    if asm_dir:
        os.makedirs(asm_dir, exist_ok=True)
        out = os.path.join(asm_dir, "libfp8gemm.so")
    try:
        objs = [os.path.join(asm_dir or work, os.path.splitext(os.path.basename(src))[0] + ".o") for src in SOURCES]
        extra = ["-save-temps=obj"] if asm_dir else []
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            jobs = [pool.submit(_run, [hipcc(), *HIPCC_FLAGS, *extra, "-c", src, "-o", obj], verbose, asm_dir)
                    for src, obj in zip(SOURCES, objs)]
            for job in jobs:
                job.result()
        tmp = out + ".tmp%d" % os.getpid()
        _run([hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", *objs, "-o", tmp], verbose)
        os.replace(tmp, out)
    finally:
        shutil.rmtree(work, ignore_errors=True)
    return out


if __name__ == "__main__":
    asm = None
    if "--asm" in sys.argv:
        asm = os.path.join(ROOT, "_build", "asm")
    print(build(asm_dir=asm, verbose=True))
