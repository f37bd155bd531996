"""When the compiled binding is built again, and what a failure of that leaves (no GPU needed)."""

import os

import pytest

from programmable_block_sparse_b200 import build as b


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A binding of its own beside the built library; the compiler is counted, not run."""
    b.build()
    monkeypatch.setattr(b, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "BINDING_STAMP", str(tmp_path / "binding.stamp"))
    runs = []

    def compiled():
        runs.append(1)
        open(b.BINDING_PATH, "w").close()

    monkeypatch.setattr(b, "_build_binding", compiled)
    return runs


def test_another_torch_or_interpreter_builds_the_binding_again(place, monkeypatch):
    b.build()
    b.build()
    assert len(place) == 1
    monkeypatch.setattr(b, "_binding_key", lambda: "torch 0.0, another\n")
    assert not b._binding_is_current()
    b.build()
    b.build()
    assert len(place) == 2 and b._binding_is_current()


def test_a_binding_older_than_its_source_is_built_again(place):
    b.build()
    os.utime(b.BINDING_PATH, (1, 1))
    b.build()
    assert len(place) == 2


def test_without_a_binding_the_library_is_built_all_the_same(place, monkeypatch, capfd):
    """Headers that are missing cost the calls of the binding, not the others, and
    never leave a binding of another ABI behind."""
    b.build()
    monkeypatch.setattr(b, "_binding_key", lambda: "torch 0.0, another\n")

    def fails():
        raise RuntimeError("g++ failed for binding.cpp: no Python.h")

    monkeypatch.setattr(b, "_build_binding", fails)
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert not os.path.exists(b.BINDING_PATH) and "no Python.h" in capfd.readouterr().err
