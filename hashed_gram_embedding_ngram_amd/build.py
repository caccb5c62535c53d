"""Build libngram.so in-tree with hipcc for gfx950.

Flags: -O3; -ffp-contract=off so that every fp32 add and multiply stays the
single IEEE operation written in the source (the gate's fused multiply-add is
an explicit fmaf); packed fp32 instructions disabled (the kernels need none).
"""
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "ngram.hip")
SOURCES = [SRC] + [os.path.join(HERE, "csrc", f) for f in ("norm8.hip", "project8.hip", "adamw8.hip", "int4.hip", "beam8.hip",
                                                               "distill8.hip")]
LIB = os.path.join(HERE, "libngram.so")
ARCH = os.environ.get("NGRAM_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    "-O3", f"--offload-arch={ARCH}", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def build(verbose: bool = False, extra=()) -> str:
    """Compile every source to an object file (at once, one process each) and
    link them."""
    with tempfile.TemporaryDirectory(dir=HERE, prefix="_build_") as tmp:
        objects, running = [], []
        for src in SOURCES:
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            cmd = ["hipcc", *HIPCC_FLAGS, *extra, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            objects.append(obj)
            running.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
        logs = [p.communicate()[0] for p in running]
        link = ["hipcc", f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", LIB + ".tmp", *objects]
        if all(p.returncode == 0 for p in running):
            r = subprocess.run(link, capture_output=True, text=True)
            logs.append(r.stdout + r.stderr)
        if any(p.returncode for p in running) or r.returncode != 0:
            sys.stderr.write("".join(logs))
            raise RuntimeError("hipcc failed to build libngram.so")
        if "-Rpass-analysis=kernel-resource-usage" in extra:
            sys.stdout.write("".join(logs))
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
