"""The build and the import where the binding module of the operators around the token mixers is missing, or
was built for another Python or torch; no GPU."""
import importlib.util
import os
import shutil
import subprocess
import sys
import types

import pytest

import linear_attention_attn_b200 as la

PKG = os.path.dirname(la.__file__)


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build script with its products in a folder of their own and nothing to compile but the module."""
    spec = importlib.util.spec_from_file_location("la_b200_build_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "OBJ", str(tmp_path))
    monkeypatch.setattr(mod, "LIB", str(tmp_path / "libla_b200.so"))
    monkeypatch.setattr(mod, "BIND", str(tmp_path / "_la_bind.so"))
    monkeypatch.setattr(mod, "_sources", lambda: [mod.BIND_SRC])
    monkeypatch.setattr(mod, "_compile", lambda src, verbose: src)
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(mod, "subprocess", types.SimpleNamespace(run=run))
    mod.calls = calls
    return mod


def test_import_without_the_binding_module(tmp_path):
    pkg = tmp_path / "linear_attention_attn_b200"
    pkg.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), pkg)
    os.symlink(os.path.join(PKG, "libla_b200.so"), pkg / "libla_b200.so")
    code = ("import linear_attention_attn_b200 as la, torch\n"
            "assert la.__file__.startswith(%r)\n"
            "assert la.la_workspace_size('bidir_fwd', 1, 2, 64, 64, torch.float16) > 0\n"
            "try:\n    la.la_group_norm_fwd(torch.zeros(1, 2, 4), torch.zeros(1, 2, 4), 2)\n"
            "except ImportError as e:\n    assert '_la_bind.so' in str(e) and 'build.py' in str(e)\n"
            "else:\n    raise AssertionError('no ImportError')\n" % str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code], cwd=str(tmp_path), capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr


def test_the_library_builds_without_what_only_the_module_needs(build, monkeypatch, capsys):
    assert build._bind_missing() == ""
    with monkeypatch.context() as m:
        m.setattr(build, "find_spec", lambda name: None)
        assert build._bind_missing() == "torch"
        assert build.build() == build.LIB
        assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)
        assert "torch not found" in capsys.readouterr().err
        m.setattr(build, "shutil", types.SimpleNamespace(which=lambda name: None))
        assert build._bind_missing() == "g++"
    build.build()
    assert os.path.exists(build.BIND)


def test_a_module_for_another_torch_is_built_again(build, monkeypatch):
    build.build()
    n = len(build.calls)
    build.build()
    assert len(build.calls) == n                          # nothing has changed
    monkeypatch.setattr(build, "_bind_for", lambda: "another")
    os.utime(build.BIND, (1, 1))
    build.build()
    assert [c[0] for c in build.calls[n:]] == ["g++", "g++"]          # compiled and linked
