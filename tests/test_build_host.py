"""What build() does about the optional modules, with a compiler that is not there or fails."""
import os
import re
from types import SimpleNamespace

import pytest

import paged_kv_decode_host_gb300 as pkd
from paged_kv_decode_host_gb300 import _build, drafts


@pytest.fixture
def modules(tmp_path, monkeypatch):
    """build() with its optional modules in a folder of their own and a recorded compiler."""
    pkd.build()
    calls, works = [], {"cc": True, "c++": True}

    def run(command, **kw):
        name = os.path.basename(command[0])
        calls.append(name)
        assert name in works, "the library is built already"
        if works[name]:
            open(command[command.index("-o") + 1], "w").close()
        return SimpleNamespace(returncode=0 if works[name] else 1, stdout="", stderr="no such library")

    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(_build, "PYPLAN", str(tmp_path / "_pkd_plan.so"))
    monkeypatch.setattr(_build, "PYSTEP", str(tmp_path / "_pkd_step.so"))
    monkeypatch.setattr(_build, "_python_include", lambda: "/include")
    monkeypatch.setattr(_build, "_torch_dir", lambda: "/torch")
    monkeypatch.setattr(_build.shutil, "which", lambda name: "/usr/bin/" + name)
    monkeypatch.setattr(_build.subprocess, "run", run)
    return SimpleNamespace(calls=calls, works=works, plan=tmp_path / "_pkd_plan.so", step=tmp_path / "_pkd_step.so")


def test_modules_are_built_once(modules):
    pkd.build()
    assert sorted(modules.calls) == ["c++", "cc"] and modules.plan.exists() and modules.step.exists()
    pkd.build()
    assert len(modules.calls) == 2


def test_a_module_that_cannot_be_built_builds_nothing_else_again(modules, capsys):
    modules.works["c++"] = False
    modules.step.write_text("an old one")
    pkd.build()
    assert not modules.step.exists() and "not built" in capsys.readouterr().err   # nor stays the old one
    pkd.build()
    pkd.build()
    assert sorted(modules.calls) == ["c++", "cc"]


def test_another_torch_or_a_missing_file_builds_a_module_anew(modules, monkeypatch):
    pkd.build()
    modules.calls.clear()
    monkeypatch.setattr(_build.shutil, "which", lambda name: "/opt/bin/" + name)
    pkd.build()
    assert modules.calls == []   # (a compiler elsewhere is no reason)
    monkeypatch.setattr(_build, "_torch_version", lambda: "0.0.1")
    pkd.build()
    assert sorted(modules.calls) == ["c++", "cc"]
    os.remove(modules.plan)
    pkd.build()
    assert modules.calls.count("cc") == 2 and modules.calls.count("c++") == 1


def test_without_a_compiler(modules, monkeypatch):
    modules.step.write_text("built elsewhere")
    monkeypatch.setattr(_build.shutil, "which", lambda name: None)
    pkd.build()
    assert modules.calls == [] and modules.step.exists() and not modules.plan.exists()


def test_modules_of_other_entry_points_or_another_torch_are_not_used(monkeypatch):
    torch = pytest.importorskip("torch")
    with open(os.path.join(_build.INCLUDE, "pkd.h")) as f:
        assert int(re.search(r"#define PKD_STEP_ABI (\d+)", f.read())[1]) == drafts.STEP_ABI
    pkd.build()
    if not os.path.exists(_build.PYSTEP):
        pytest.skip("no compiled calls on tensors here")
    m = pytest.importorskip("paged_kv_decode_host_gb300._pkd_step")
    version = torch.__version__.split("+")[0]
    for args in ((drafts.STEP_ABI + 1, version), (drafts.STEP_ABI, "0.0.1")):
        with pytest.raises(ImportError):
            m.init(*args, 0, 0, 0)
    monkeypatch.setattr(drafts, "_step_module", None)
    assert drafts._step() is not None
    monkeypatch.setattr(drafts, "STEP_ABI", drafts.STEP_ABI + 1)
    monkeypatch.setattr(drafts, "_step_module", None)
    assert drafts._step() is None   # and every call takes the general path
