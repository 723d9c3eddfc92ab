"""The build of the token mixers' marshaller: it never stands in the way of the library, and a binary of another Python
or torch is not loaded."""
import os

import pytest


@pytest.fixture()
def B(tmp_path, monkeypatch):
    from routed_expert_ffn_iq2_b200 import build

    build.build()
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    return build


@pytest.fixture()
def native(monkeypatch):
    from routed_expert_ffn_iq2_b200 import _native

    monkeypatch.setattr(_native, "_marshal_mod", None)
    return _native


def test_a_compiler_that_fails_costs_the_mixers_alone(B, native, monkeypatch):
    monkeypatch.setattr(B, "CXX", "false")
    with pytest.warns(UserWarning, match="token mixers"):
        assert B.build() == B.LIB
    native.lib()
    with pytest.raises(RuntimeError, match="not built"):
        native._marshal()
    monkeypatch.setattr(B, "CXX", str(B.MARSHAL) + ".no-such-compiler")
    with pytest.warns(UserWarning, match="token mixers"):
        assert B.build() == B.LIB
    with pytest.raises((RuntimeError, OSError)):
        B.build_marshal()


def test_a_binary_of_another_torch_is_built_again(B, native, monkeypatch):
    calls = []

    def compiler(cmd, **kw):
        calls.append(cmd)
        abi = next(a for a in cmd if a.startswith("-DREDLITE_MARSHAL_ABI="))
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("binary redlite_marshal_abi:" + abi.split("=", 1)[1].strip('"') + "; binary")
        return type("R", (), {"returncode": 0, "stdout": b""})()

    monkeypatch.setattr(B.subprocess, "run", compiler)
    B.build_marshal()
    assert len(calls) == 1 and os.path.exists(B.MARSHAL) and B.marshal_abi_matches()
    B.build_marshal()
    assert len(calls) == 1
    import torch

    monkeypatch.setattr(torch, "__version__", "9.9")
    assert not B.marshal_abi_matches()
    with pytest.raises(RuntimeError, match="another Python or torch"):
        native._marshal()
    B.build_marshal()
    assert len(calls) == 2 and B.marshal_abi_matches()
    # a build that does not go through leaves nothing that counts as current
    monkeypatch.setattr(torch, "__version__", "9.8")
    monkeypatch.setattr(B.subprocess, "run", lambda cmd, **kw: type("R", (), {"returncode": 1, "stdout": b"no"})())
    with pytest.warns(UserWarning, match="token mixers"):
        B.build()
    monkeypatch.setattr(torch, "__version__", "9.9")
    assert not B.marshal_abi_matches()
    assert not os.path.exists(B.MARSHAL)


def test_the_library_is_built_without_torch(B, monkeypatch):
    import sys

    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="token mixers"):
        assert B.build() == B.LIB


def test_the_binary_tells_what_it_was_built_against():
    from routed_expert_ffn_iq2_b200 import build

    build.build()
    assert build.marshal_abi_matches()
