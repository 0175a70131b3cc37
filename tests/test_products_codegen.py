"""The generated gfx950 code of the products and of the transposed compress (hipcc, no GPU needed):
no packed float32 arithmetic, no spilled registers in the kernels, m0 written only by the
loads to LDS that are written as asm, and the waits that those need."""
import importlib.util
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_compression_tensor_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")


def flags():
    spec = importlib.util.spec_from_file_location(
        "_tfp8_lib_build", os.path.join(ROOT, "fp8_compression_tensor_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return [f for f in mod.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]


@pytest.fixture(scope="module", params=["tfp8_matmul.hip", "tfp8_compress_t.hip"])
def kernels(request, tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "k.s")
    r = subprocess.run(["hipcc", *flags(), "--cuda-device-only", "-S", "-o", out,
                        os.path.join(CSRC, request.param)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    bodies = {}
    for m in re.finditer(r"^(_ZN4tfp8\w*k_\w+):.*?s_endpgm", text, re.S | re.M):
        bodies[m.group(1)] = m.group(0).split("\n")
    spills = re.findall(r"\.vgpr_spill_count:\s*(\d+)", text)
    return request.param, bodies, spills


def test_every_kernel_was_found(kernels):
    name, bodies, spills = kernels
    want = ["k_matmul_tile", "k_matmul_split"] if "matmul" in name else ["k_compress_t"]
    assert all(any(w in b for b in bodies) for w in want) and len(spills) == len(bodies)


def test_no_packed_float32_and_no_spills(kernels):
    _, bodies, spills = kernels
    for name, body in bodies.items():
        assert not [l for l in body if re.search(r"v_pk_(add|mul|fma)_f32", l)], name
    assert all(int(s) == 0 for s in spills), spills


def test_m0_is_written_only_for_the_loads_that_follow(kernels):
    _, bodies, _ = kernels
    for name, body in bodies.items():
        code = [l.split(";")[0].strip() for l in body]
        code = [l for l in code if l and not l.startswith(".") and not l.endswith(":")]
        for i, l in enumerate(code):
            if re.search(r"\bm0\b", l):
                assert l.startswith("s_mov_b32 m0, s") and code[i + 1] == "s_nop 0", (name, l)
                assert re.match(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], s\d+ offen lds",
                                code[i + 2]), (name, code[i + 2])
            if " lds" in l:
                assert code[i - 2].startswith("s_mov_b32 m0"), (name, l)
