"""The package's names are the binding's, at every look-up. No GPU."""
import os
import subprocess
import sys

import rank_gradient_sketching_sketch_amd as L
from rank_gradient_sketching_sketch_amd import binding as B


def test_names_are_the_bindings():
    for name in L.__all__:
        assert getattr(L, name) is getattr(B, name), name


def test_a_replacement_in_the_binding_shows(monkeypatch):
    for name in ("logra_route", "logra_grad_clip", "AdamWList"):
        first = getattr(L, name)
        other = object()
        monkeypatch.setattr(B, name, other)
        assert getattr(L, name) is other
        monkeypatch.undo()
        assert getattr(L, name) is first


def test_what_a_caller_puts_into_the_package_stays(monkeypatch):
    mine = object()
    L.logra_route
    monkeypatch.setattr(L, "logra_route", mine)
    monkeypatch.setattr(B, "logra_grad_clip", object())
    assert L.logra_route is mine and L.logra_grad_clip is B.logra_grad_clip


def test_a_binding_loaded_anew_shows():
    """In a process of its own: other modules hold the binding's classes."""
    code = """
import importlib, sys
sys.path.insert(0, %r)
import rank_gradient_sketching_sketch_amd as L
old = L.logra_route, L.LograError
from rank_gradient_sketching_sketch_amd import binding as B
importlib.reload(B)
assert L.logra_route is B.logra_route is not old[0] and L.LograError is B.LograError
del B.logra_route
assert not hasattr(L, "logra_route") and hasattr(L, "logra_grad_clip") and not hasattr(L, "nothing")
"""
    root = os.path.dirname(os.path.dirname(L.__file__))
    subprocess.run([sys.executable, "-c", code % root], check=True, timeout=120)
