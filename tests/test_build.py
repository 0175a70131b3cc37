"""The build where the module that g++ makes cannot be made: the library is there all the same."""
import os
import shutil
import subprocess

import pytest

from fp8_compression_tensor_amd import build

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")


@pytest.mark.parametrize("command", [["false"], ["no-such-compiler"], None])
def test_the_library_needs_no_module(tmp_path, monkeypatch, command):
    source = tmp_path / "one.hip"
    source.write_text("#include <hip/hip_runtime.h>\n__global__ void k(int *p) { *p = 1; }\n"
                      'extern "C" int one() { return 1; }\n')

    def rows_command(out):
        if command is None:
            raise ImportError("no torch")
        return command

    monkeypatch.setattr(build, "SOURCES", [str(source)])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "ROWS", str(tmp_path / "_rows.so"))
    monkeypatch.setattr(build, "rows_command", rows_command)
    (tmp_path / "_rows.so").write_text("of an older library")
    with pytest.raises(RuntimeError, match="grad_norm and adamw"):
        build.build()
    assert "one" in subprocess.run(["nm", "-D", str(tmp_path / "lib.so")], capture_output=True, text=True).stdout
    assert not os.path.exists(tmp_path / "_rows.so")
