"""When the serving operators' Python extension is built, and what happens where it cannot be (no compiler runs here)."""
import os
import types

import pytest
import torch

from asymmetric_head_kv_b200 import build as b


@pytest.fixture
def sandbox(monkeypatch, tmp_path):
    """The extension's files in a folder of the test's own, and a compiler that only notes its calls."""
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_serving.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "BINDING_KEY", str(tmp_path / "objects" / "serving.key"), raising=False)
    monkeypatch.setattr(b, "subprocess", types.SimpleNamespace(run=run))
    return calls


def test_built_once_and_again_for_another_torch_or_python(sandbox, monkeypatch):
    assert b._build_binding(False) == b.BINDING and len(sandbox) == 1
    assert b._build_binding(False) == b.BINDING and len(sandbox) == 1
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert b._build_binding(False) == b.BINDING and len(sandbox) == 2
    monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: False)
    b._build_binding(False)
    assert len(sandbox) == 3 and "-D_GLIBCXX_USE_CXX11_ABI=0" in sandbox[-1]
    real = b.sysconfig.get_config_var
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda n: "cpython-other" if n == "SOABI" else real(n))
    b._build_binding(False)
    b._build_binding(False)
    assert len(sandbox) == 4
    b._build_binding(True)
    assert len(sandbox) == 5


@pytest.mark.parametrize("lacks", ["g++", "headers"])
def test_the_library_does_not_wait_for_what_the_extension_needs(sandbox, monkeypatch, tmp_path, lacks):
    real = b.shutil.which
    if lacks == "g++":
        monkeypatch.setattr(b.shutil, "which", lambda n: None if n == "g++" else real(n))
    else:
        paths = dict(b.sysconfig.get_paths(), include=str(tmp_path / "none"))
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: paths)
    built = []
    monkeypatch.setattr(b, "_build_one", lambda lib, *a: built.append(lib) or lib)
    with pytest.warns(UserWarning, match="missing"):
        assert b.build() == b.LIB
    assert built == [b.LIB, b.LIB_CHECKED] and not sandbox and not os.path.exists(b.BINDING)


def test_a_failing_compiler_is_an_error(sandbox, monkeypatch):
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: types.SimpleNamespace(returncode=1, stdout="", stderr="no"))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b._build_binding(False)
