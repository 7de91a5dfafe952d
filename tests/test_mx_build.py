"""The Python binding of the microscaled calls is optional, and taken only where it was built for this torch and this
Python."""
import os
import sys
import sysconfig
import types

import pytest

import qlora_parameter_efficient_b200 as q
from qlora_parameter_efficient_b200 import build


@pytest.fixture()
def unloaded(monkeypatch):
    """As before the first microscaled call."""
    build.build_library()
    monkeypatch.setattr(q, "_bind", None)
    monkeypatch.setattr(q, "_bind_looked_for", False)


def test_named_after_what_it_is_built_for(monkeypatch):
    import torch
    name = os.path.basename(q._mx_bind_path())
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name and name.endswith(".so")
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert os.path.basename(q._mx_bind_path()) != name
    assert os.path.dirname(build.build_library()) == os.path.dirname(q._mx_bind_path())


def test_one_of_another_torch_is_not_taken(monkeypatch, unloaded):
    import torch
    build.build_binding()
    assert q._binding() is not None
    monkeypatch.setattr(q, "_bind", None)
    monkeypatch.setattr(q, "_bind_looked_for", False)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert q._binding() is None


def test_one_that_cannot_be_loaded_is_as_none(monkeypatch, unloaded, tmp_path):
    bad = tmp_path / "_mx_bind-bad.so"
    bad.write_bytes(b"not a shared object")
    monkeypatch.setattr(q, "_mx_bind_path", lambda: str(bad))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert q._binding() is None
    import torch
    with pytest.raises(ValueError):                          # the longer way's own checks
        q.mxfp4_quantize(torch.zeros(4, 64))


def test_the_library_builds_without_torch(monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)          # `import torch` raises ImportError
    assert os.path.exists(build.build_library())
    assert build.build_binding() is None and "not built" in capsys.readouterr().out


def test_no_headers(monkeypatch, capsys, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", types.SimpleNamespace(__file__=str(tmp_path / "__init__.py")))
    assert build.build_binding() is None and "not built" in capsys.readouterr().out
