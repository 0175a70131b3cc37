"""Build the gfx950 HIP library libtfp8.so in-tree with hipcc, and with g++ the CPython module _rows.so,
which reads tensors' properties for the binding."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtfp8.so")
ROWS = os.path.join(HERE, "_rows.so")
SOURCES = [os.path.join(CSRC, f) for f in
           ("tfp8_kernels.hip", "tfp8_compress_t.hip", "tfp8_matmul.hip", "tfp8_optimizer.hip",
            "tfp8_moe.hip")]

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


def rows_command(out: str) -> list[str]:
    import torch

    at = os.path.dirname(torch.__file__)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f"-I{at}/include", f"-I{at}/include/torch/csrc/api/include",
            f"-I{sysconfig.get_paths()['include']}", "-o", out, os.path.join(CSRC, "tfp8_rows.cpp"),
            f"-L{at}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(verbose: bool = False, extra: list[str] | None = None, out: str | None = None) -> str:
    """The library at `out`; without it in the package, and the module beside it."""
    with_rows = out is None
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
            raise RuntimeError(f"{cmd[0]} failed ({r.returncode}):\n{err}")
        if verbose and err.strip():
            print(err, file=sys.stderr)

    # one object a source, side by side, then the link
    flags = [*(f for f in HIPCC_FLAGS if f != "-shared"), *(extra or [])]
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        jobs = [["hipcc", *flags, "-c", "-o", o, s] for s, o in zip(SOURCES, objects)]
        with ThreadPoolExecutor(len(jobs) + 1) as pool:
            rows = pool.submit(lambda: run(rows_command(ROWS + ".tmp"))) if with_rows else None
            list(pool.map(run, jobs))
        run(["hipcc", "--offload-arch=gfx950", "-shared", "-o", tmp, *objects])
    os.replace(tmp, out)
    if with_rows:
        try:
            rows.result()
        except Exception as e:  # no g++, no headers of Python or torch: the rest works without
            if os.path.exists(ROWS):  # an older library's
                os.remove(ROWS)
            raise RuntimeError(f"{out} is built, the module _rows.so is not, which grad_norm and adamw need: "
                               f"{e}") from e
        os.replace(ROWS + ".tmp", ROWS)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
