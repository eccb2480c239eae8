"""What is rebuilt when: the library alone, and the binding for the torch and Python that load it.  No GPU needed."""
import os

import pytest

from sparse_state_linear_sdm_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_binding()


def test_what_was_just_built_is_current():
    assert build.up_to_date() and build.binding_up_to_date()


def test_a_binding_of_another_torch_or_python_is_stale(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "_binding_tag", lambda: "another torch")
    assert not build.binding_up_to_date()
    monkeypatch.undo()
    monkeypatch.setattr(build, "BINDING_TAG", str(tmp_path / "none"))
    assert not build.binding_up_to_date()


def test_the_tag_names_torch_and_python(monkeypatch):
    import sys

    import torch

    assert torch.__version__ in build._binding_tag() and sys.version in build._binding_tag()
    before = build._binding_tag()
    monkeypatch.setattr(torch, "__version__", "0.0")
    assert build._binding_tag() != before


def test_the_library_is_built_without_the_binding(monkeypatch, tmp_path):
    """No torch headers and no host compiler are needed for it."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')

    def none(*_):
        raise AssertionError("the binding is not the library's")

    monkeypatch.setattr(build, "_sources", lambda: [str(src)])
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "absent.so"))
    for name in ("_compile_binding", "_link_binding"):
        monkeypatch.setattr(build, name, none)
    assert build.build() == str(tmp_path / "lib.so") and os.path.exists(tmp_path / "lib.so")
    assert not os.path.exists(build.BINDING)


def test_the_library_does_not_age_with_the_binding(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "absent.so"))
    assert build.up_to_date() and not build.binding_up_to_date()
