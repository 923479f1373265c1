"""The build of the FP8 calls' marshalling module: one for each interpreter, and the library without it where it
cannot be made."""

import os
import sysconfig

import pytest

from moe_prefill_nvfp4_gb300 import _lib, build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The library is built; the module goes to a folder of its own and counts as missing."""
    build.build()
    target = tmp_path / "call.so"
    monkeypatch.setattr(build, "call_path", lambda: str(target))
    return target


def test_the_module_belongs_to_one_interpreter():
    assert os.path.basename(build.call_path()).endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert sysconfig.get_config_var("SOABI") in build.call_path()


@pytest.mark.parametrize("compiler", ["no-such-compiler", "false"], ids=["missing", "failing"])
def test_the_library_does_not_need_the_module(elsewhere, monkeypatch, compiler):
    monkeypatch.setenv("CC", compiler)
    elsewhere.write_text("of older sources")
    os.utime(elsewhere, (1, 1))
    before = os.path.getmtime(build.lib_path())
    with pytest.warns(RuntimeWarning, match="no FP8 calls"):
        assert build.build() == build.lib_path()
    assert os.path.getmtime(build.lib_path()) == before  # not built again for the module's sake
    assert not elsewhere.exists()  # an old module would call a library that is newer
    assert not build.up_to_date()


def test_fp8_calls_say_why(elsewhere, monkeypatch):
    monkeypatch.setenv("CC", "no-such-compiler")
    monkeypatch.setattr(_lib, "_FP8", None)
    with pytest.raises(RuntimeError, match="no-such-compiler"):
        _lib._fp8()
    assert _lib._FP8 is None


def test_the_module_alone_is_built(elsewhere):
    before = os.path.getmtime(build.lib_path())
    assert not build.up_to_date()
    build.build()
    assert elsewhere.exists() and build.up_to_date()
    assert os.path.getmtime(build.lib_path()) == before
