"""What the build makes where parts of its surroundings are missing or have changed. Needs no GPU."""
import os
import time

import pytest

import attention_flash_gqa_gb300 as attn
from attention_flash_gqa_gb300 import _build


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A build of one source into a folder of its own."""
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "OPS", str(tmp_path / "_ops.so"))
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path / "tmp"))
    monkeypatch.setattr(_build, "OPS_TAG", str(tmp_path / "tmp" / "tag.txt"), raising=False)
    monkeypatch.setattr(_build, "SOURCES", ["merge_lse.cu"])
    return tmp_path


@pytest.mark.parametrize("missing", ["compiler", "headers"])
def test_library_without_the_binding(place, monkeypatch, missing):
    """No g++, or torch's headers are not there: the C library is linked, the build says what is missing."""
    run = _build.subprocess.run

    def fail(cmd, *args, **kw):
        if cmd[0] != "g++":
            return run(cmd, *args, **kw)
        if missing == "compiler":
            raise FileNotFoundError("g++")
        return run([cmd[0], "-fsyntax-only", "-x", "c++", "-include", "no/such/header.h", os.devnull], *args, **kw)

    monkeypatch.setattr(_build.subprocess, "run", fail)
    with pytest.raises(RuntimeError, match="py_ops.cpp"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.OPS)


def test_library_without_torch(place, monkeypatch):
    """There is nothing to bind: the library alone is the whole build."""
    monkeypatch.setattr(_build, "torch_tag", lambda: None)
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB) and not os.path.exists(_build.OPS)
    assert _build.up_to_date()


def test_binding_of_another_torch_is_built_again(place, monkeypatch):
    """File times do not tell that torch was changed."""
    os.makedirs(_build.BUILD_DIR)
    for f in (_build.LIB, _build.OPS):
        open(f, "w").close()
        os.utime(f, (time.time() + 60,) * 2)
    with open(_build.OPS_TAG, "w") as f:
        f.write("torch 1.0 for another python")
    assert not _build.up_to_date()
    built = []

    def ops():
        built.append("ops")
        with open(_build.OPS_TAG, "w") as f:
            f.write(_build.torch_tag())

    monkeypatch.setattr(_build, "_build_ops", ops)
    monkeypatch.setattr(_build, "_build_lib", lambda verbose: built.append("lib"), raising=False)
    _build.build()
    assert built == ["ops"] and _build.up_to_date()
    _build.build()
    assert built == ["ops"]


def test_binding_of_another_torch_is_not_loaded(monkeypatch):
    """The calls through it refuse, by name, what would not fit."""
    _build.build()
    monkeypatch.setattr(attn, "_bound", None)
    monkeypatch.setattr(_build, "ops_tag", lambda: "torch 1.0 for another python", raising=False)
    with pytest.raises(RuntimeError, match="torch 1.0 for another python"):
        attn.attn_qk_norm_rope(None, None, None, None, None, None)
