"""The build's dependencies, with compilers that are fakes: the C library needs nvcc alone."""
import os
import subprocess

import pytest

from polynomial_matrix_whitening_gb300 import build as B


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """Compilers that write an empty result, in a folder of their own; fails: the tools that fail."""
    class Fake:
        fails, ran = (), []

        def run(self, cmd, **_):
            tool, out = os.path.basename(cmd[0]), cmd[cmd.index("-o") + 1]
            self.ran.append(tool)
            if tool in self.fails:
                return subprocess.CompletedProcess(cmd, 1, "", "no")
            open(out, "w").close()
            return subprocess.CompletedProcess(cmd, 0, "", "")
    f = Fake()
    f.ran = []
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libanvil.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_anvil_binding.so"))
    monkeypatch.setattr(B, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(B.subprocess, "run", f.run)
    return f


def test_library_without_pytorch(fake, monkeypatch):
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: None)
    assert os.path.exists(B.build()) and not os.path.exists(B.BINDING)
    assert "g++" not in fake.ran


def test_library_with_a_pytorch_without_cuda(fake, monkeypatch, tmp_path):
    class Spec:
        submodule_search_locations = [str(tmp_path / "torch")]
    os.makedirs(tmp_path / "torch" / "lib")
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: Spec)
    assert os.path.exists(B.build()) and not os.path.exists(B.BINDING)
    assert "g++" not in fake.ran


def test_library_before_a_binding_that_fails(fake):
    pytest.importorskip("torch")
    if B.binding_command() is None:
        pytest.skip("a PyTorch without CUDA")
    fake.fails = ("g++",)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed on .*binding.cpp"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    fake.fails = ()
    del fake.ran[:]
    B.build()  # only what is missing
    assert os.path.exists(B.BINDING) and fake.ran == ["g++"]


def test_a_library_source_that_fails(fake):
    fake.fails = ("nvcc",)
    with pytest.raises(RuntimeError, match="nvcc failed on"):
        B.build()
    assert not os.path.exists(B.LIB)
