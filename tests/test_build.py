"""The extension module beside the library: made for one PyTorch and Python, and not needed by the library."""
import os

import pytest
import torch

from qwen3_decoder_transformer_gb300 import binding
from qwen3_decoder_transformer_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def test_nothing_is_built_twice(monkeypatch):
    monkeypatch.setattr(B, "_build_tensors", lambda: pytest.fail("built again"))
    monkeypatch.setattr(B.subprocess, "run", lambda *a, **k: pytest.fail("compiled again"))
    assert B.build() == B.LIB


@pytest.mark.parametrize("change", ["version", "place", "python"])
def test_another_torch_or_python_has_a_module_of_its_own(monkeypatch, change):
    made = []
    monkeypatch.setattr(B, "_build_tensors", lambda: made.append(1))
    if change == "version":
        monkeypatch.setattr(torch, "__version__", torch.__version__ + ".1")
    elif change == "place":
        monkeypatch.setattr(torch, "__file__", "/elsewhere/torch/__init__.py")
    else:
        ours = B.sysconfig.get_config_var
        monkeypatch.setattr(B.sysconfig, "get_config_var", lambda n: ".other.so" if n == "EXT_SUFFIX" else ours(n))
    B.build()
    assert made == [1]
    # and the one that is there is not loaded
    monkeypatch.setattr(binding, "_tensors", None)
    with pytest.raises(RuntimeError, match="not built for this PyTorch"):
        binding._checks()


def test_the_library_is_built_without_the_module(monkeypatch, tmp_path):
    """A compiler that fails, and one that is missing: the library is built, with a warning that says why."""
    monkeypatch.setattr(B, "tensors_path", lambda: str(tmp_path / "none.so"))
    linked = []
    monkeypatch.setattr(B, "_fresh", lambda path: False)
    monkeypatch.setattr(B, "_build_library", lambda verbose: linked.append(1))
    for error in (RuntimeError("no Python.h"), FileNotFoundError("g++")):
        def fail(error=error):
            raise error

        monkeypatch.setattr(B, "_build_tensors", fail)
        with pytest.warns(RuntimeWarning, match=str(error)):
            assert B.build() == B.LIB
    assert linked == [1, 1] and os.path.exists(B.LIB)
