"""The compiled argument marshalling is rebuilt, and refused, when Python or torch is another than it was built
against (no GPU, no compiler needed)."""
from __future__ import annotations

import os

import pytest

from calibration_free_weight_dualquant_b200 import binding, build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Modules go to a folder of its own; commands are recorded and write their output file instead of running."""
    ran = []

    def run(cmd, what):
        ran.append(what)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)
        return ""

    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_dq_torch.so"), raising=False)
    monkeypatch.setattr(build, "_run", run)
    return ran


def test_rebuilt_for_another_torch(tree, monkeypatch):
    import torch

    first = build.build_marshal()
    assert build.build_marshal() == first and len(tree) == 1 and os.path.exists(first)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build_marshal()
    assert len(tree) == 2
    build.build_marshal()
    assert len(tree) == 2


def test_rebuilt_for_another_python(tree, monkeypatch):
    build.build_marshal()
    real = build.sysconfig.get_config_var
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda k: "cpython-00-other" if k == "SOABI" else real(k))
    build.build_marshal()
    assert len(tree) == 2


def test_loading_one_of_another_torch_is_refused(monkeypatch):
    import torch

    build.build()
    monkeypatch.setattr(binding, "_marshal", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(binding.DQError) as e:
        binding.load_marshal()
    assert e.value.status == 5 and "not built" in str(e.value)


def test_the_library_is_built_where_the_module_cannot_be(tmp_path, monkeypatch):
    """No Python headers, say: the solver is built and stays usable, the linear layer's calls say what is missing."""
    def run(cmd, what):
        if "dq_torch" in what:
            raise RuntimeError(what + " failed")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)
        return ""

    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libdq.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_dq_torch.so"), raising=False)
    monkeypatch.setattr(build, "_run", run)
    with pytest.warns(UserWarning, match="linear layer"):
        assert build.build() == str(tmp_path / "libdq.so")
    assert os.path.exists(tmp_path / "libdq.so")
    with pytest.raises(RuntimeError):
        build.build_marshal()
    monkeypatch.setattr(binding, "_marshal", None)
    with pytest.raises(binding.DQError) as e:
        binding.load_marshal()
    assert e.value.status == 5 and "not built" in str(e.value)
