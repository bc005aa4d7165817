"""When the library and the front end count as built (CPU)."""
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
