"""The library's calls do not hang on the binding's fast path: where that is missing, broken or
another torch's, they are checked in Python."""
import os
import warnings

import pytest
import torch

import paged_fp8_kv_03_gb300 as pkv
from paged_fp8_kv_03_gb300 import build
from tests.test_fp8b_host import test_binding_refuses


@pytest.fixture
def fresh(monkeypatch):
    """As before the first load()."""
    monkeypatch.setattr(pkv, "_lib", None)
    monkeypatch.setattr(pkv, "_fast", None)
    return monkeypatch


def _works():
    assert pkv.pkv_version() > 0 and pkv.pkv_decode_noalloc_scratch_bytes() > 0
    assert pkv.pkv_prefill_fp8b_workspace_size(1, 1, 1, 100) > 0
    with pytest.raises(ValueError):
        pkv.kv_append_fp8(torch.zeros(1, 1, 128), None, None, None, None, None, None)
    test_binding_refuses()


def test_missing(fresh, tmp_path):
    fresh.setattr(build, "BINDING", str(tmp_path / "none.so"))
    with pytest.warns(RuntimeWarning, match="fast path"):
        pkv.load()
    _works()


def test_broken(fresh, tmp_path):
    path = tmp_path / "broken.so"
    path.write_bytes(b"no library")
    fresh.setattr(build, "BINDING", str(path))
    with pytest.warns(RuntimeWarning, match="fast path"):
        pkv.load()
    _works()


def test_the_one_that_was_built(fresh):
    """It is named by the torch that it was built with, so another one is not taken for it."""
    assert torch.__version__ in os.path.basename(build.BINDING)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        pkv.load()
    assert pkv._fast is not pkv._NoFast
    _works()


@pytest.mark.parametrize("compiles", [False, True])
def test_a_binding_that_cannot_be_built_leaves_the_library(monkeypatch, tmp_path, capsys, compiles):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "_stale", lambda target, files: target == build.BINDING)
    monkeypatch.setattr(build, "_binding_commands", lambda: (["true" if compiles else "false"], ["false"], str(tmp_path / "tmp.so")))
    assert build.build() == build.LIB
    assert "cannot be built" in capsys.readouterr().err and not os.path.exists(build.BINDING)
