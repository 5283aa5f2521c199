"""The C library's build needs no torch: where torch is absent the module of the Python calls is left out."""
import importlib.util

from clebsch_gordan_tensor_cgtp_amd import build as libbuild


def test_the_python_calls_are_left_out_without_torch(monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(libbuild, "_compile", lambda args: (_ for _ in ()).throw(AssertionError("compiled")))
    assert libbuild.build_calls() is None
    assert "torch" in capsys.readouterr().err
