"""What is built for whom (nothing is compiled here)."""
import os
import subprocess
import sys

import pytest

from combine_persistent_warp_gb300 import build, native

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def no_binding(monkeypatch, tmp_path):
    """A machine without the headers that _ops.so needs, the library up to date."""
    def refuse():
        raise RuntimeError("no headers")

    monkeypatch.setattr(build, "OPS", str(tmp_path / "_ops.so"))
    monkeypatch.setattr(build, "_compile_binding", refuse)
    monkeypatch.setattr(build, "library_up_to_date", lambda: True)


def test_the_layer_loads_where_the_operators_module_cannot_be_built(no_binding, monkeypatch):
    monkeypatch.setattr(native, "_lib", None)
    assert native.load() is not None
    assert not os.path.exists(build.OPS)


def test_building_everything_or_the_module_says_what_is_missing(no_binding):
    for f in (build.build, build.build_binding):
        with pytest.raises(RuntimeError, match="no headers"):
            f()


def test_the_module_does_not_wait_for_the_kernels_sources(monkeypatch, tmp_path):
    made = tmp_path / "_ops.so"
    made.touch()
    (tmp_path / "_ops.so.for").write_text(build._built_against())
    monkeypatch.setattr(build, "OPS", str(made))
    monkeypatch.setattr(build, "library_up_to_date", lambda: False)
    assert build.binding_up_to_date() and not build.up_to_date()


def test_the_package_imports_without_the_operators():
    code = "import sys, combine_persistent_warp_gb300 as p; p.load(); assert not any(m.endswith('._ops') for m in sys.modules)"
    assert subprocess.run([sys.executable, "-c", code], cwd=ROOT).returncode == 0


def test_a_module_built_for_another_pytorch_is_not_up_to_date(monkeypatch, tmp_path):
    made = tmp_path / "_ops.so"
    made.touch()
    monkeypatch.setattr(build, "OPS", str(made))
    assert not build.binding_up_to_date()                # of unknown origin
    (tmp_path / "_ops.so.for").write_text(build._built_against())
    assert build.binding_up_to_date()
    import torch
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    assert not build.binding_up_to_date()
