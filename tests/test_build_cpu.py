"""The build of the binding's extension: what is left of it when a step fails,
and which one the binding takes."""
import os

import pytest

import mixture_experts_layer_mm_gb300._lib as binding
from mixture_experts_layer_mm_gb300 import buildlib


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's own files under a temporary folder, with an earlier extension."""
    monkeypatch.setattr(buildlib, "BUILD", str(tmp_path))
    monkeypatch.setattr(buildlib, "MARSHAL", str(tmp_path / "_marshal.so"))
    (tmp_path / "_marshal.so").write_bytes(b"built from other sources")
    return tmp_path


def test_an_extension_that_does_not_compile_leaves_no_earlier_one(elsewhere, monkeypatch, capsys):
    monkeypatch.setenv("CXX", "/bin/false")
    obj = buildlib._compile_marshal()
    assert obj is None and "not built" in capsys.readouterr().out
    buildlib._link_marshal(obj)
    assert os.listdir(elsewhere) == []
    buildlib._link_marshal(None)  # nothing there to remove


def test_an_extension_that_does_not_link_leaves_no_earlier_one(elsewhere, mmlib, capsys):
    bad = elsewhere / "marshal.cpp.o"
    bad.write_bytes(b"no object")
    buildlib._link_marshal(str(bad))
    assert "not built" in capsys.readouterr().out
    assert os.listdir(elsewhere) == ["marshal.cpp.o"]


def test_an_extension_is_linked_again_for_another_object(elsewhere, mmlib, monkeypatch):
    # Sources that went back to an earlier state: its object is the older file.
    monkeypatch.setenv("CXX", "/bin/true")
    for name in ("a.o", "b.o"):
        (elsewhere / name).write_bytes(b"")
        os.utime(elsewhere / name, (0, 0))
    linked = []
    for name in ("a.o", "a.o", "b.o", "a.o"):
        (elsewhere / "_marshal.so.tmp").write_bytes(name.encode())
        buildlib._link_marshal(str(elsewhere / name))
        linked.append((elsewhere / "_marshal.so").read_bytes().decode())
    assert linked == ["a.o", "a.o", "b.o", "a.o"]


@pytest.mark.parametrize("changed", ["MARSHAL_SRC", "MARSHAL_HEADER"])
def test_the_tag_follows_the_sources(changed, tmp_path, monkeypatch):
    before = buildlib.marshal_tag()
    other = tmp_path / "other"
    with open(getattr(buildlib, changed), "rb") as f:
        other.write_bytes(f.read() + b"\n")
    monkeypatch.setattr(buildlib, changed, str(other))
    assert buildlib.marshal_tag() != before


def test_the_binding_declines_an_extension_of_other_sources(mmlib, monkeypatch):
    if binding._load_fast() is None:
        pytest.skip("the extension is not built")
    monkeypatch.setattr(buildlib, "marshal_tag", lambda: "other")
    assert binding._load_fast() is None
