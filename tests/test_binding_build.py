"""_binding.so is never one of another source, torch or Python: built again, or not there."""
import os
import types

import pytest


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """The build script, whose outputs lie in a folder of their own."""
    import __graft_entry__
    mod = __graft_entry__._builder()
    monkeypatch.setattr(mod, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(mod, "BUILD", str(tmp_path / "_build"))
    os.makedirs(mod.BUILD)
    return mod


@pytest.fixture
def moe():
    import __graft_entry__
    __graft_entry__._builder().build()
    import fp8_grouped_expert_x128_gb300 as lib
    return lib


def compiler(tmp_path, works):
    """Stands for g++: writes what it was called with to its output, or fails."""
    path = tmp_path / ("works" if works else "fails")
    path.write_text('#!/bin/sh\nout=\nfor a in "$@"; do [ "$out" = next ] && echo "$@" > "$a"; out=; [ "$a" = -o ] && out=next; done\nexit 0\n'
                    if works else "#!/bin/sh\nexit 1\n")
    path.chmod(0o755)
    return str(path)


def test_what_cannot_be_built_again_goes(builder, tmp_path, monkeypatch, capsys):
    monkeypatch.setenv("CXX", compiler(tmp_path, False))
    with open(builder.BINDING, "w") as f:
        f.write("of an older source")
    os.utime(builder.BINDING, (1, 1))
    builder._build_binding("/usr/local/cuda", False)
    assert not os.path.exists(builder.BINDING)
    assert "not built" in capsys.readouterr().err


def test_what_nothing_is_there_to_build_with_goes(builder, monkeypatch, capsys):
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(builder.shutil, "which", lambda name: None)
    with open(builder.BINDING, "w") as f:
        f.write("of an older source")
    os.utime(builder.BINDING, (1, 1))
    builder._build_binding("/usr/local/cuda", False)
    assert not os.path.exists(builder.BINDING)
    assert "not built" in capsys.readouterr().err


def test_another_torch_or_python_builds_it_again(builder, tmp_path, monkeypatch):
    monkeypatch.setenv("CXX", compiler(tmp_path, True))
    builder._build_binding("/usr/local/cuda", False)

    def built_again():
        os.utime(builder.BINDING, (2 ** 31, 2 ** 31))          # newer than all sources
        builder._build_binding("/usr/local/cuda", False)
        return os.path.getmtime(builder.BINDING) != 2 ** 31

    assert not built_again()
    with monkeypatch.context() as m:
        m.setattr(builder.importlib.metadata, "version", lambda name: "0.0.1")
        assert built_again()
    assert built_again()                                        # and back
    with monkeypatch.context() as m:
        m.setattr(builder.sys, "version", "4.0")
        assert built_again()
    assert built_again() and not built_again()


def test_one_of_another_layout_is_not_taken(moe):
    assert moe._native is not None and moe._is_ours(moe._native)
    made = moe._native.made_for()
    for i in range(len(made)):
        other = list(made)
        other[i] += 1
        assert not moe._is_ours(types.SimpleNamespace(made_for=lambda: tuple(other)))
    assert not moe._is_ours(types.SimpleNamespace())            # of before it could be asked
    assert not moe._is_ours(types.SimpleNamespace(made_for=lambda: made + (0,)))
