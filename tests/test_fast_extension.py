"""The marshalling extension is the one built for the running torch, and its absence is said (CPU)."""
import os
import shutil
import sys

import pytest
import torch

from ragged_attention_token_gb300 import build, rra


@pytest.fixture(scope="module")
def L():
    build.build()
    return rra.lib()


def test_built_and_loaded(L):
    path = build.fast_path()
    assert torch.__version__ in os.path.basename(path) and sys.implementation.cache_tag in os.path.basename(path)
    assert build._fast_up_to_date()
    assert rra._FAST is not None and os.path.samefile(rra._FAST.__file__, path)


def test_one_built_against_another_torch_is_not_used(L, monkeypatch):
    assert build._fast_up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert not build._fast_up_to_date()
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        assert rra._load_fast(L) is None


def test_a_file_that_does_not_load_is_said(L, monkeypatch, tmp_path):
    bad = tmp_path / "_rra_fast.so"
    bad.write_bytes(b"not a library")
    monkeypatch.setattr(build, "fast_path", lambda: str(bad))
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        assert rra._load_fast(L) is None


def test_a_failed_build_leaves_no_older_extension(L, monkeypatch, tmp_path):
    path = tmp_path / "_rra_fast.so"
    shutil.copy(build.fast_path(), path)
    monkeypatch.setattr(build, "fast_path", lambda: str(path))
    monkeypatch.setattr(build, "FAST_SRC", str(tmp_path / "no_such_source.cpp"))
    with pytest.raises(RuntimeError):
        build.build_fast(force=True)
    assert not path.exists()
