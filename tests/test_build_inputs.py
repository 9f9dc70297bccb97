"""When the compiled parts count as up to date."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def build():
    import __graft_entry__
    __graft_entry__.build()
    from bwd_dw_column_gb300 import _build
    return _build


def test_another_torch_or_interpreter_builds_the_module_anew(build, monkeypatch):
    """_cake_block.so is compiled against torch's C++ headers: file times alone do not say that it fits."""
    import sys
    assert build.up_to_date()
    for where, name, value in ((torch, "__version__", "0.0.1"), (torch, "__file__", "/elsewhere/torch/__init__.py"),
                               (sys, "version", "3.0")):
        with monkeypatch.context() as m:
            m.setattr(where, name, value)
            assert not build.up_to_date(), name
    assert build.up_to_date()


def test_a_changed_source_builds_anew(build, monkeypatch, tmp_path):
    newer = tmp_path / "newer.cuh"
    newer.write_text("")
    later = os.path.getmtime(build.LIB) + 10
    os.utime(newer, (later, later))
    files = build._inputs()
    with monkeypatch.context() as m:
        m.setattr(build, "_inputs", lambda: files + [str(newer)])
        assert not build.up_to_date()
    assert build.up_to_date()
