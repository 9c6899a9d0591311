"""CPU checks of the build: what is put in place when a step of it fails, and which file of
compiled calls is loaded.  No compiler runs here."""
import os
import sys

import pytest
import torch

import expert_layer_moe_amd as moe
from expert_layer_moe_amd import binding, build as b


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A folder of an older build, and compilers that write what they were to make."""
    monkeypatch.setattr(b, "LIBDIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmoe_amd.so"))
    monkeypatch.setattr(b, "_run", lambda cmd, verbose, noise="": open(cmd[cmd.index("-o") + 1], "w").write("new"))
    (tmp_path / "libmoe_amd.so").write_text("old")
    (tmp_path / os.path.basename(b.calls_path())).write_text("old")
    (tmp_path / "_moe_calls.so").write_text("older")
    return tmp_path


def _there(place):
    return {p.name: p.read_text() for p in place.iterdir() if not p.name.endswith(".tmp")}


def test_both_are_put_in_place(place):
    b.build()
    assert _there(place) == {"libmoe_amd.so": "new", os.path.basename(b.calls_path()): "new"}


@pytest.mark.parametrize("failing", ["libmoe_amd.so", "_moe_calls"])
def test_nothing_changes_where_a_step_fails(place, monkeypatch, failing):
    before, run = _there(place), b._run

    def fail(cmd, verbose, noise=""):
        if failing in cmd[cmd.index("-o") + 1]:
            raise RuntimeError("does not compile")
        run(cmd, verbose, noise)
    monkeypatch.setattr(b, "_run", fail)
    with pytest.raises(RuntimeError, match="does not compile"):
        b.build()
    assert _there(place) == before


@pytest.mark.parametrize("lacking", ["compiler", "headers"])
def test_the_library_is_built_without_what_the_calls_need(place, monkeypatch, lacking):
    """And no calls of an older library stay beside it."""
    if lacking == "compiler":
        monkeypatch.setattr(b, "host_cxx", lambda: None)
    else:
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(place)})
    with pytest.warns(UserWarning, match="Python calls"):
        b.build()
    assert _there(place) == {"libmoe_amd.so": "new"}


def test_calls_are_those_of_this_interpreter_and_torch(place, monkeypatch):
    name = os.path.basename(b.calls_path())
    assert sys.implementation.cache_tag in name and torch.__version__ in name
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert os.path.basename(b.calls_path()) != name


def test_missing_calls_are_named_by_the_first_one(tmp_path, monkeypatch):
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(binding, "CALLS_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="none.so is missing.*this interpreter and torch"):
        moe.moe_quant_mxfp4(torch.zeros(1, 32))
    moe.load_library()   # (the others do not ask for them)
    with pytest.raises(ValueError):
        moe.moe_quant_fp8(torch.zeros(1, 32))
