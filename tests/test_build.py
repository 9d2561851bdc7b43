"""What build() builds, and what it says when it cannot. No GPU, and nothing is compiled here beyond what is missing."""
import pytest

from shared_kv_draft_b200 import build as b
from shared_kv_draft_b200 import orthrus


def test_a_failing_command_is_named():
    with pytest.raises(RuntimeError, match=r"^g\+\+ failed"):
        b._run(["g++", "no-such-file.cpp"], False)


def test_the_binding_follows_torch(monkeypatch):
    b.build()
    assert b.up_to_date()
    monkeypatch.setattr(b, "_binding_tag", lambda: "torch 0.0, other")
    assert b.library_up_to_date() and not b.binding_up_to_date() and not b.up_to_date()


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    b.build()
    assert orthrus._native().built_for == b._binding_tag()
    monkeypatch.setattr(orthrus, "_binding", None)
    monkeypatch.setattr(b, "_binding_tag", lambda: "torch 0.0, other")
    with pytest.raises(ImportError, match="built for torch"):
        orthrus._native()


def test_the_library_stands_without_the_binding(monkeypatch):
    """Without Python's headers the library is still built and its path returned; the failure is a warning."""
    b.build()
    monkeypatch.setattr(b, "binding_up_to_date", lambda: False)
    monkeypatch.setattr(b, "_build_binding", lambda verbose: b._run(["g++", "no-such-file.cpp"], verbose))
    with pytest.warns(UserWarning, match="native binding is not"):
        assert b.build() == b.LIB
    assert b.library_up_to_date()


def test_the_library_stands_without_torch(monkeypatch):
    def absent():
        raise ImportError("no torch")

    b.build()
    monkeypatch.setattr(b, "_binding_tag", absent)
    with pytest.warns(UserWarning, match="no torch"):
        assert b.build() == b.LIB


def test_a_failing_library_raises(monkeypatch):
    monkeypatch.setattr(b, "library_up_to_date", lambda: False)
    monkeypatch.setattr(b, "_compile", lambda *a: b._run(["g++", "no-such-file.cpp"], False))
    with pytest.raises(RuntimeError):
        b.build()
