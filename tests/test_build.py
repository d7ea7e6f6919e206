"""The build in a folder of its own: the library needs the CUDA toolkit alone, the binding torch."""
import os
import subprocess
import sys

import pytest

from sparse_global_attention_b200 import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUN = """
import sys
sys.path.insert(0, {root!r})
{hide}
from sparse_global_attention_b200 import build as b
b.CSRC = {at!r}
b.BUILD, b.LIB, b.BINDING = {at!r} + "/build", {at!r} + "/lib.so", {at!r} + "/binding.so"
b.build()
"""


def run(at, hide):
    (at / "one.cu").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    return subprocess.run([sys.executable, "-c", RUN.format(root=ROOT, at=str(at), hide=hide)], capture_output=True, text=True)


@pytest.mark.parametrize("missing", ["torch", "torch.utils.cpp_extension"])
def test_library_without_torch(tmp_path, missing):
    r = run(tmp_path, f"sys.modules[{missing!r}] = None")
    assert r.returncode == 0, r.stderr
    assert (tmp_path / "lib.so").exists() and not (tmp_path / "binding.so").exists()
    assert "lib.so is built" in r.stderr and "binding.so" in r.stderr and "torch" in r.stderr


def test_binding_that_does_not_compile_leaves_the_library(tmp_path):
    (tmp_path / "torch_binding.cpp").write_text("no C++\n")
    r = run(tmp_path, "")
    assert r.returncode != 0 and "g++ failed on torch_binding.cpp" in r.stderr
    assert (tmp_path / "lib.so").exists() and not (tmp_path / "binding.so").exists()


def test_binding_takes_the_string_type_of_the_installed_torch(tmp_path, monkeypatch):
    """std::string has two forms in GCC's library; torch's build says which one its symbols take."""
    import torch
    seen = []

    def fake(cmd, **kw):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(b.subprocess, "run", fake)
    for abi in (True, False):
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", abi)
        b.build_binding()
        assert f"-D_GLIBCXX_USE_CXX11_ABI={int(abi)}" in seen[-1]
