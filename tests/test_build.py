"""The build: a binding follows the PyTorch and Python it links against, and a
binding that does not compile does not keep the library from being linked.
One small source in a folder of its own; no GPU."""
import os

import pytest

from paged_kv_cache_mapping_gb300 import build as b


@pytest.fixture
def small(tmp_path, monkeypatch):
    for name, file in (("BUILD", "objs"), ("LIB", "lib.so"), ("BINDING", "binding.so"), ("BINDING_FOR", "objs/binding_for.txt")):
        monkeypatch.setattr(b, name, str(tmp_path / file))
    monkeypatch.setattr(b, "SOURCES", ["pkv_append.cu"])
    monkeypatch.setattr(b, "binding_command", lambda out: ["touch", out])  # g++ is not what is tested
    return tmp_path


def test_a_binding_follows_what_it_links_against(small, monkeypatch):
    made = []
    monkeypatch.setattr(b, "binding_command", lambda out: made.append(out) or ["touch", out])
    b.build()
    assert os.path.exists(b.LIB) and os.path.exists(b.BINDING) and len(made) == 1
    b.build()
    assert len(made) == 1
    monkeypatch.setattr(b, "binding_target", lambda: "another PyTorch")
    b.build()
    assert len(made) == 2
    b.build()
    assert len(made) == 2
    os.remove(b.BINDING_FOR)
    b.build()
    assert len(made) == 3


def test_the_target_names_python_and_pytorch():
    import sys

    import torch
    t = b.binding_target()
    assert sys.version in t and torch.__version__ in t and os.path.dirname(torch.__file__) in t


def test_the_library_is_linked_without_the_binding(small, monkeypatch, capfd):
    monkeypatch.setattr(b, "binding_command", lambda out: ["false"])
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
    monkeypatch.setattr(b, "binding_command", lambda out: ["touch", out])
    assert b.build() == b.LIB and os.path.exists(b.BINDING)
