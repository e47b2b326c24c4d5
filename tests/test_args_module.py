"""The native argument checks are an extra: a module built for another torch or Python is not used, one that cannot be
built is not left behind, and the library is built without it."""
import importlib.machinery
import importlib.util
import os
import pathlib
import shutil

import pytest
import torch

from fp8_block_scaled_amd import build

HERE = os.path.exists(build.ARGS)


def load(path):
    loader = importlib.machinery.ExtensionFileLoader("_args", str(path))
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_args", loader))
    loader.exec_module(module)
    return module


@pytest.mark.skipif(not HERE, reason="the argument checks are not built here")
def test_is_not_loaded_beside_another_torch(tmp_path, monkeypatch):
    for name in ("first", "second"):
        shutil.copy(build.ARGS, tmp_path / f"{name}.so")
    assert load(tmp_path / "first.so").address(None, (), (), 0) is None
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    with pytest.raises(ImportError, match="built for torch"):
        load(tmp_path / "second.so")


@pytest.mark.parametrize("step", [None, ["false"], ["/no/such/compiler"]])
def test_an_old_module_does_not_stay(step, tmp_path, monkeypatch):
    old = tmp_path / "_args.so"
    old.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "ARGS", str(old))
    monkeypatch.setattr(build, "_args_step", lambda out: step)
    if step is None:
        assert build.build_args() is False
    else:
        with pytest.warns(UserWarning, match="argument checks"):
            assert build.build_args() is False
    assert os.listdir(tmp_path) == []


def test_a_built_module_takes_the_old_ones_place(tmp_path, monkeypatch):
    old = tmp_path / "_args.so"
    old.write_bytes(b"old")
    monkeypatch.setattr(build, "ARGS", str(old))
    monkeypatch.setattr(build, "_args_step", lambda out: ["cp", __file__, out])
    assert build.build_args() is True and old.read_bytes() == pathlib.Path(__file__).read_bytes() and os.listdir(tmp_path) == ["_args.so"]


def test_the_library_is_built_where_the_checks_are_not(tmp_path, monkeypatch):
    """build() with compilers that only write their output."""
    def ran(cmd, **kw):
        class Result:
            returncode, stdout, stderr = int(cmd[0] == "broken"), "", ""
        if not Result.returncode:
            pathlib.Path(cmd[cmd.index("-o") + 1]).write_text("built")
        return Result

    monkeypatch.setattr(build.subprocess, "run", ran)
    monkeypatch.setattr(build, "_hipcc", lambda: "hipcc")
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgfg.so"))
    monkeypatch.setattr(build, "ARGS", str(tmp_path / "_args.so"))
    monkeypatch.setattr(build, "_args_step", lambda out: ["broken", "-o", out])
    with pytest.warns(UserWarning, match="argument checks"):
        assert build.build() == str(tmp_path / "libgfg.so")
    assert (tmp_path / "libgfg.so").exists() and not (tmp_path / "_args.so").exists()
