"""When the extension module is built again, and that a stale one is refused (CPU)."""
import importlib
import os

import pytest


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build with its outputs in a folder of its own and a compiler that writes an empty file."""
    from frame_sparse_attention_b200 import build as b
    monkeypatch.setattr(b, "BIND", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(b, "BIND_BUILT_FOR", str(tmp_path / "built_for"))
    b.runs = []

    def compile_(args):
        b.runs.append(args)
        open(args[args.index("-o") + 1], "w").close()
    monkeypatch.setattr(b.subprocess, "check_call", compile_)
    yield b
    del b.runs


def _count(build, force=False):
    n = len(build.runs)
    build._build_bind(build._nvcc(), force)
    return len(build.runs) - n


def test_the_module_is_built_again_for_another_torch_or_interpreter(build, monkeypatch):
    import torch
    assert _count(build) == 1 and _count(build) == 0
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "9.9.9")
        assert _count(build) == 1 and _count(build) == 0
    assert _count(build) == 1 and _count(build) == 0
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399")
        assert _count(build) == 1
    assert _count(build) == 1 and _count(build) == 0


def test_the_module_is_built_again_when_something_is_missing_or_newer(build):
    assert _count(build) == 1
    os.remove(build.BIND)
    assert _count(build) == 1 and _count(build) == 0
    os.remove(build.BIND_BUILT_FOR)  # a module that nobody can say what it was built for
    assert _count(build) == 1 and _count(build) == 0
    os.utime(build.BIND, (1, 1))     # older than its source
    assert _count(build) == 1 and _count(build) == 0
    assert _count(build, force=True) == 1


def test_a_module_of_another_torch_is_refused(monkeypatch):
    import torch
    from frame_sparse_attention_b200 import _cache
    monkeypatch.setattr(_cache, "_bind", None)
    assert _cache._load_bind().built_for.startswith("torch ")
    monkeypatch.setattr(_cache, "_bind", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.raises(RuntimeError, match="build it with"):
        _cache._load_bind()
    assert _cache._bind is None


def test_a_module_that_does_not_load_is_refused(monkeypatch):
    from frame_sparse_attention_b200 import _cache
    monkeypatch.setattr(_cache, "_bind", None)

    def fail(name, package):
        raise ImportError("undefined symbol")
    monkeypatch.setattr(importlib, "import_module", fail)
    with pytest.raises(RuntimeError, match="undefined symbol.*build it with"):
        _cache._load_bind()
