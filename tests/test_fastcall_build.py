"""The compiled marshalling belongs to one torch and one Python: it is rebuilt for another, and one built for another
is not loaded."""
import os
import shutil
import subprocess
import sysconfig

import pytest

from attn_fwd_02_gb300 import binding, build


@pytest.fixture(scope="module")
def built():
    torch = pytest.importorskip("torch")
    out = build._compile_fastcall()
    if out is None:
        pytest.skip("fastcall.cpp cannot be compiled here")
    return torch, out


def test_named_by_the_installed_torch_and_python(built):
    torch, out = built
    assert build._installed_torch()[1] == torch.__version__
    assert out == build.fastcall_path(torch.__version__) and os.path.exists(out)
    assert torch.__version__ in os.path.basename(out) and out.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_loaded_for_its_own_torch_alone(built):
    torch, out = built
    m = binding._load_fastcall(torch.__version__, torch.compiled_with_cxx11_abi())
    assert m is not None and m.torch_version == torch.__version__
    assert binding._load_fastcall(torch.__version__, not torch.compiled_with_cxx11_abi()) is None
    other = torch.__version__.split("+")[0] + "+other"  # the same number, another build
    assert binding._load_fastcall(other, torch.compiled_with_cxx11_abi()) is None
    try:  # a file that bears the wrong name
        shutil.copy(out, build.fastcall_path(other))
        assert binding._load_fastcall(other, torch.compiled_with_cxx11_abi()) is None
    finally:
        os.remove(build.fastcall_path(other))


def test_rebuilt_when_torch_changes(built, monkeypatch):
    folder = build._installed_torch()[0]
    monkeypatch.setattr(build, "_installed_torch", lambda: (folder, "9.9.9+other"))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("compiled")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    out = build.fastcall_path("9.9.9+other")
    try:
        assert build._compile_fastcall() == out and os.path.exists(out)
        assert '-DATTN_TORCH_VERSION="9.9.9+other"' in ran[0]
        assert build._compile_fastcall() == out and len(ran) == 1  # current from then on
    finally:
        os.remove(out)


def test_without_torch(monkeypatch, capsys):
    monkeypatch.setattr(build, "_installed_torch", lambda: ("", ""))
    assert build._compile_fastcall() is None
    assert "Python" in capsys.readouterr().err
