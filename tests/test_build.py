"""What is built when: the library by itself, the calls' module beside it (no compiler runs here)."""
import os
import subprocess

import pytest

from paged_kv_cache_377_b200 import _binding, build, tree


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """The build's outputs in a folder of their own, and compilers that only note their commands; ``broken`` commands fail."""
    tree._lib()                                      # the real one is loaded, whatever happens below
    commands, broken = [], []
    for name, file in (("LIB", "libpagedkv.so"), ("MARSHAL", "_marshal.so"), ("MARSHAL_ABI", "_marshal.abi"),
                       ("BUILD", "_build")):
        monkeypatch.setattr(build, name, str(tmp_path / file), raising=False)

    def run(cmd, **_):
        commands.append(cmd)
        failed = any(b in " ".join(cmd) for b in broken)
        if not failed:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return subprocess.CompletedProcess(cmd, 1 if failed else 0, "", "broken" if failed else "")

    monkeypatch.setattr(build.subprocess, "run", run)
    return commands, broken


@pytest.mark.parametrize("what", ["marshal.cpp", "-lc10_cuda"])
def test_the_library_does_not_need_the_module(sandbox, what):
    """Without Python's headers or torch's libraries the library is built and in place all the same."""
    commands, broken = sandbox
    broken.append(what)
    build.build(force=True)
    assert os.path.exists(build.LIB) and not os.path.exists(build.MARSHAL)
    commands.clear()
    assert _binding._ensure_built() == build.LIB and not commands
    with pytest.raises(RuntimeError, match="marshal"):
        _binding._ensure_marshal()
    broken.clear()
    _binding._ensure_marshal()
    assert os.path.exists(build.MARSHAL) and not build.marshal_is_stale()


def test_nothing_is_built_twice(sandbox):
    commands, _ = sandbox
    build.build()
    build.build_marshal()
    assert len(commands) == len(build.SOURCES) + 3
    commands.clear()
    build.build()
    build.build_marshal()
    _binding._ensure_built()
    _binding._ensure_marshal()
    assert not commands


def test_another_torch_or_python_rebuilds_the_module_alone(sandbox, monkeypatch):
    commands, _ = sandbox
    build.build()
    build.build_marshal()
    for attr, value in (("__version__", "99.0"), ("compiled_with_cxx11_abi", lambda: False)):
        commands.clear()
        import torch
        monkeypatch.setattr(torch, attr, value)
        assert build.marshal_is_stale() and not build.is_stale()
        build.build()
        build.build_marshal()
        assert len(commands) == 2 and not build.marshal_is_stale()
    os.remove(build.MARSHAL_ABI)
    assert build.marshal_is_stale()


def test_only_the_calls_that_use_the_module_ask_for_it(sandbox, monkeypatch):
    """Sizes and refusals that go straight to the library work without it; a call through it raises."""
    commands, broken = sandbox
    broken.append("marshal.cpp")
    monkeypatch.setattr(tree, "_marshal", None)
    assert tree.tree_workspace_bytes(128) > 0
    assert not commands
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        tree.paged_tree_mask(None, None, None, None, 1, None)
