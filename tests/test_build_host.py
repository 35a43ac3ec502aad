"""The build's two parts on the host: the library needs no Python headers and no torch, the
module belongs to one torch and one Python."""

import os

import pytest
import torch

import block_sparse_attention_sa_gb300 as sa
from block_sparse_attention_sa_gb300 import build as b
from helpers import lib


@pytest.fixture(scope="module", autouse=True)
def built():
    lib()


def test_a_module_that_does_not_compile_leaves_the_library(monkeypatch, tmp_path, capfd):
    made = []
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "PKG", str(tmp_path))
    monkeypatch.setattr(b, "_compile_library", lambda verbose_ptxas=False: made.append(b.LIB))

    def fail():
        raise RuntimeError("Python.h: No such file")

    monkeypatch.setattr(b, "_compile_module", fail)
    assert b.build() == b.LIB and made == [b.LIB]
    assert "Python.h" in capfd.readouterr().err


def test_the_module_of_another_torch_is_neither_kept_nor_loaded(monkeypatch):
    here = b.module_path()
    assert os.path.exists(here) and not b._module_stale()
    monkeypatch.setattr(torch, "__version__", "1.2.3+other")
    assert b.module_path() != here and b._module_stale()
    monkeypatch.setattr(sa, "_BIND", None)
    with pytest.raises(FileNotFoundError, match="block_sparse_attention_sa_gb300.build"):
        sa._bind()


def test_the_module_of_another_python_is_neither_kept_nor_loaded(monkeypatch):
    here = b.module_path()
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert b.module_path() != here and b._module_stale()


def test_what_is_built_is_not_built_again(monkeypatch):
    def never(*a, **k):
        raise AssertionError("built again")

    monkeypatch.setattr(b, "_compile_library", never)
    monkeypatch.setattr(b, "_compile_module", never)
    assert b.build() == b.LIB
