"""The build where something that only the binding to torch needs is missing:
the libraries with the C ABIs need hipcc alone."""
import importlib
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
# the module, not the package's build() of the same name
build = importlib.import_module("ssim_loss_amd.build")


@pytest.fixture
def commands(monkeypatch):
    """What the build would run; nothing is run or replaced."""
    seen = []
    monkeypatch.setattr(build, "_run", lambda cmd, verbose: seen.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    return seen


def outputs(commands):
    return [os.path.basename(c[c.index("-o") + 1]).replace(".tmp", "") for c in commands]


LIBRARIES = ["libssim_loss_amd.so", "libssim_train_amd.so"]


def test_all_three_are_built(commands):
    build.build_all()
    assert [o for o in outputs(commands) if o.endswith(".so")] == [*LIBRARIES, "_bind.so"]


def test_without_torch_the_libraries_are_built(commands, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # its import fails
    build.build_all()
    assert [o for o in outputs(commands) if o.endswith(".so")] == LIBRARIES
    assert "torch" in capsys.readouterr().err
    with pytest.raises(ImportError):
        build.build_bind()


def test_with_another_torch_the_libraries_are_built(commands, monkeypatch):
    import torch

    monkeypatch.setattr(torch.version, "hip", None)
    build.build_all()
    assert [o for o in outputs(commands) if o.endswith(".so")] == LIBRARIES


def test_without_a_host_compiler_the_binding_takes_hipccs(commands, monkeypatch):
    found = build.shutil.which
    monkeypatch.setattr(build.shutil, "which",
                        lambda name, *a: None if name in ("g++", "c++") else found(name, *a))
    build.build_bind()
    assert os.path.basename(commands[-1][0]) == "amdclang++" and os.path.exists(commands[-1][0])
