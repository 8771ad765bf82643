"""The compiled binding belongs to one Python and one torch (CPU)."""
import os
import subprocess
import sys
import types

import pytest
import torch

from exact_attention_129_b200 import build as eab
from exact_attention_129_b200 import serving


def test_another_torch_does_not_load_this_binding(monkeypatch):
    # the binding is C++ against torch's headers: a stale one could end the process
    eab.build()
    here = serving.binding_path()
    assert os.path.exists(here) and torch.__version__ in os.path.basename(here)
    monkeypatch.setattr(torch, "__version__", "99.0.1+cu999")
    monkeypatch.setattr(serving, "_binding", None)
    assert serving.binding_path() != here
    with pytest.raises(ImportError, match="99.0.1.*build"):
        serving._load()


def test_another_torch_builds_a_binding_of_its_own(monkeypatch):
    eab.build()
    assert eab.build_binding() == serving.binding_path()  # up to date: nothing is compiled
    calls = []

    def run(cmd, **_):
        calls.append(cmd)
        return types.SimpleNamespace(returncode=1, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    eab.build_binding()
    assert not calls
    for name in ((torch, "__version__", "99.0.1+cu999"),
                 (sys.implementation, "cache_tag", "cpython-399")):
        with monkeypatch.context() as m:
            m.setattr(*name)
            with pytest.raises(RuntimeError, match=name[2].replace("+", r"\+")):
                eab.build_binding()
        assert any(name[2] in x for x in calls.pop())
