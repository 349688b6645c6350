"""The build script: what is built when, and what a failure leaves behind (no compiler runs here)."""
import os
import subprocess

import pytest

from long_context_sequence_all_b200 import build as B
from long_context_sequence_all_b200 import ulysses as U


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """Outputs in a folder of their own; a compiler that writes its -o file and is written down."""
    for name in ("LIB", "NATIVE", "BUILD"):
        monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        tag = [c for c in cmd if c.startswith("-DULY_BINDING_TAG=")]
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write((tag[0].split('"')[1] if tag else "").encode() + b"\0")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "_check_register_split", lambda *a: None)
    return calls


def test_the_library_is_built_where_the_binding_cannot_be(elsewhere, monkeypatch):
    def no(force=False):
        raise RuntimeError("no headers of torch")
    monkeypatch.setattr(B, "build_native", no)
    with pytest.raises(RuntimeError, match="no headers"):
        B.build()
    assert os.path.exists(B.LIB)


def test_a_binding_for_another_torch_is_built_again(elsewhere, monkeypatch):
    assert B.build_native() == B.NATIVE and len(elsewhere) == 1
    assert B.build_native() == B.NATIVE and len(elsewhere) == 1        # nothing has changed
    assert B.native_fits(B.NATIVE)
    version = B.importlib.metadata.version
    monkeypatch.setattr(B.importlib.metadata, "version", lambda name: version(name) + ".other")
    assert not B.native_fits(B.NATIVE)
    B.build_native()
    assert len(elsewhere) == 2 and B.native_fits(B.NATIVE)


def test_a_binding_for_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(U, "_native_module", None)
    monkeypatch.setattr(B, "native_tag", lambda: "ulysses binding: torch 0.0, another")
    with pytest.raises(RuntimeError, match="another torch or Python"):
        U._native()


def test_the_built_binding_is_for_this_torch():
    import torch
    assert torch.__version__ in B.native_tag() and B.native_fits()
    assert U._native().tag == B.native_tag()
