"""The build of the library and of the operators' extension module, each for
itself, with the compilers replaced (no GPU, no compilation)."""
import os

import pytest

from qwen3_dense_decoder_gb300 import buildlib


class Compiler:
    """Counts the runs of a compiler and makes the files it names."""

    def __init__(self, monkeypatch, tmp_path, ops_fail=False):
        self.runs = {"nvcc": 0, "g++": 0}
        self.ops_fail = ops_fail
        for name, f in (("LIB", "libq3.so"), ("OPS", "_ops.so"), ("BUILD", "_build")):
            monkeypatch.setattr(buildlib, name, str(tmp_path / f))
        monkeypatch.setattr(buildlib, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
        monkeypatch.setattr(buildlib.subprocess, "run", self.run)

    def run(self, cmd, **kw):
        host = not cmd[0].endswith("nvcc")
        self.runs["g++" if host else "nvcc"] += 1

        class Result:
            returncode, stdout, stderr = (1, "", "Python.h: No such file or directory") if host and self.ops_fail else (0, "", "")
        if Result.returncode == 0:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return Result


def test_the_library_is_built_without_the_extension(monkeypatch, tmp_path, capsys):
    c = Compiler(monkeypatch, tmp_path, ops_fail=True)
    assert buildlib.build() == buildlib.LIB and os.path.exists(buildlib.LIB) and not os.path.exists(buildlib.OPS)
    assert "Python.h" in capsys.readouterr().err
    n = c.runs["nvcc"]
    assert n == len(buildlib.SOURCES) + 1
    assert buildlib.build() == buildlib.LIB                # what is missing is tried again, and that alone
    assert c.runs == {"nvcc": n, "g++": 2}


def test_operators_without_their_extension_say_why(monkeypatch):
    import builtins

    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    q3.lib()
    real = builtins.__import__

    def refuse(name, globals=None, locals=None, fromlist=(), level=0):
        if level == 1 and "_ops" in (fromlist or ()):
            raise ImportError("undefined symbol: a_name_of_another_torch")
        return real(name, globals, locals, fromlist, level)
    monkeypatch.setattr(q3, "_native", None)
    monkeypatch.setattr(builtins, "__import__", refuse)
    with pytest.raises(RuntimeError, match="a_name_of_another_torch"):
        q3.op_token_logprobs(None)


def test_the_extension_is_rebuilt_for_another_torch_or_python(monkeypatch, tmp_path):
    c = Compiler(monkeypatch, tmp_path)
    buildlib.build()
    buildlib.build()
    assert c.runs == {"nvcc": len(buildlib.SOURCES) + 1, "g++": 1}         # up to date
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "__init__.py").write_text("")
    (torch / "version.py").write_text("__version__ = '9.9'\n")
    real = buildlib.importlib.util.find_spec
    spec = type("Spec", (), {"origin": str(torch / "__init__.py")})
    monkeypatch.setattr(buildlib.importlib.util, "find_spec", lambda name: spec if name == "torch" else real(name))
    buildlib.build()
    buildlib.build()
    assert c.runs["g++"] == 2
    (torch / "version.py").write_text("__version__ = '9.10'\n")            # the same place, another version
    buildlib.build()
    assert c.runs["g++"] == 3
    ext = buildlib.sysconfig.get_config_var
    monkeypatch.setattr(buildlib.sysconfig, "get_config_var", lambda n: ".cpython-399.so" if n == "EXT_SUFFIX" else ext(n))
    buildlib.build()
    buildlib.build()
    assert c.runs == {"nvcc": len(buildlib.SOURCES) + 1, "g++": 4}         # the library needs neither
