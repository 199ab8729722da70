"""Build libgdr.so (the HIP kernels and the C ABI) in-tree for gfx950."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(HERE, "libgdr.so")
# csrc: the gated delta rule; csrc_ops: the operators around it in a layer
SOURCES = ["csrc/gdr_api.cpp", "csrc/gdr_fwd.hip", "csrc/gdr_bwd.hip", "csrc/gdr_recurrent.hip",
           "csrc_ops/ops_api.cpp", "csrc_ops/conv1d.hip", "csrc_ops/rms_norm.hip",
           "csrc_ops/gated_norm.hip", "csrc_ops/sandwich_norm.hip", "csrc_ops/quantize.hip",
           "csrc_ops/int8_matmul.hip",
           "csrc_ops/ssm_fwd.hip", "csrc_ops/ssm_bwd.hip", "csrc_ops/ssm_bwd_bf16.hip",
           "csrc_ops/ssm_bwd_fp16.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(line for line in res.stdout.splitlines() if "packed-fp32-ops" not in line)
    if res.returncode != 0:
        sys.stderr.write(out + "\n")
        raise RuntimeError("hipcc failed (%d)" % res.returncode)
    if verbose and out.strip():
        print(out, flush=True)


def build(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as work:
        objs = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1)) as pool:
            for f in [pool.submit(_run, [hipcc] + HIPCC_FLAGS + ["-c", "-o", o, os.path.join(HERE, s)],
                                  verbose) for s, o in zip(SOURCES, objs)]:
                f.result()
        _run([hipcc] + HIPCC_FLAGS + ["-shared", "-o", tmp] + objs, verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
