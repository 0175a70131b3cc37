"""Build the gfx950 HIP library libtfp8.so in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtfp8.so")
SOURCES = [os.path.join(CSRC, f) for f in
           ("tfp8_kernels.hip", "tfp8_compress_t.hip", "tfp8_matmul.hip")]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # float arithmetic exactly as written: no contraction of a*b+c into fma, no fast math
    "-ffp-contract=off",
    "-fno-fast-math",
    # keep the compiler from emitting packed FP32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def build(verbose: bool = False, extra: list[str] | None = None, out: str | None = None) -> str:
    out = out or LIB
    tmp = out + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        # hipcc's host pass does not know the packed-fp32 feature name; that warning is expected
        noise = "is not a recognized feature for this target"
        err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed ({r.returncode}):\n{err}")
        if verbose and err.strip():
            print(err, file=sys.stderr)

    # one object a source, side by side, then the link
    flags = [*(f for f in HIPCC_FLAGS if f != "-shared"), *(extra or [])]
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            list(pool.map(run, (["hipcc", *flags, "-c", "-o", o, s]
                                for s, o in zip(SOURCES, objects))))
        run(["hipcc", "--offload-arch=gfx950", "-shared", "-o", tmp, *objects])
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
