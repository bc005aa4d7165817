"""When the library and the front end count as built, and what each needs (CPU)."""
import os
import re
import subprocess
import sys

import pytest
import torch

from causal_attention_fwd_attn_b200 import _lib, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_a_front_end_for_another_torch_is_neither_current_nor_loaded(monkeypatch):
    assert build.up_to_date() and build.front_built_for() == build.front_tag()
    assert str(torch.__version__) in build.front_tag()
    _lib.front()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    monkeypatch.setattr(_lib, "_front", None)
    assert not build.up_to_date()
    with pytest.raises(RuntimeError, match=r"0\.0\.0\+other.*causal_attention_fwd_attn_b200\.build"):
        _lib.front()
    # only the front end is built again
    done = []
    monkeypatch.setattr(build, "_run", lambda cmd, what, *a, **k: done.append(what) or 1 / 0)
    with pytest.raises(ZeroDivisionError):
        build.build()
    assert done == ["g++"]


def test_a_file_that_carries_no_tag_is_not_current(monkeypatch, tmp_path):
    other = tmp_path / "_front.so"
    other.write_bytes(b"something else")
    monkeypatch.setattr(build, "FRONT", str(other))
    assert build.front_built_for() is None and not build.up_to_date()
    monkeypatch.setattr(build, "FRONT", str(tmp_path / "missing.so"))
    assert build.front_built_for() is None and not build.up_to_date()


def test_the_library_needs_no_torch(tmp_path):
    """build.py by itself, where torch cannot be imported: the library, and a word about the rest."""
    code = ("import sys; sys.modules['torch'] = None; sys.path.insert(0, sys.argv[1]); import build; "
            "build.FRONT = sys.argv[2]; print(build.build()); "
            "ran = []; build._run = lambda cmd, what, *a, **k: ran.append(what); "
            "build.os.replace = lambda *a: None; build.build(force=True); print(ran)")
    run = subprocess.run([sys.executable, "-c", code, build.PKG, str(tmp_path / "_front.so")],
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    assert run.stdout.split("\n")[:2] == [build.LIBRARY, "['nvcc']"]
    assert "_front.so is not built: no torch" in run.stderr
    assert not os.path.exists(tmp_path / "_front.so")


@pytest.mark.parametrize("missing,said", [("ATen.h", "torch's headers"), ("libc10_cuda.so", "torch with CUDA"),
                                          ("Python.h", "Python's headers"), ("g++", "g\\+\\+")])
def test_a_front_end_that_cannot_be_built_is_left_out(monkeypatch, capsys, tmp_path, missing, said):
    exists, which = os.path.exists, build.shutil.which
    monkeypatch.setattr(build, "FRONT", str(tmp_path / "_front.so"))
    monkeypatch.setattr(build.os.path, "exists", lambda p: exists(p) and os.path.basename(p) != missing)
    monkeypatch.setattr(build.shutil, "which", lambda p: None if p == missing else which(p))
    monkeypatch.setattr(build, "_build_front", lambda verbose: 1 / 0)
    assert build.up_to_date() and build.build() == build.LIBRARY
    monkeypatch.setattr(build, "up_to_date", lambda: False)
    assert build.build() == build.LIBRARY
    monkeypatch.undo()
    assert re.search("not built: no " + said, capsys.readouterr().err)
    # its functions say that it is missing
    monkeypatch.setattr(build, "FRONT", str(tmp_path / "_front.so"))
    monkeypatch.setattr(_lib, "_front", None)
    with pytest.raises(RuntimeError, match="is not built"):
        _lib.front()
