"""The CPython module of the linear-attention calls is theirs alone: without it the rest is built and
runs."""
import sys

import pytest
import torch

import gated_delta_rule_rgdr_amd as rg


def test_other_calls_do_without_the_module(monkeypatch):
    monkeypatch.setattr(rg, "_lib", None)
    monkeypatch.setattr(rg, "_quick", None)
    monkeypatch.delattr(rg, "_la_binding", raising=False)
    monkeypatch.setitem(sys.modules, rg.__name__ + "._la_binding", None)  # its import raises
    assert rg.status_string(0) == "RGDR_OK"
    with pytest.raises(RuntimeError, match="on the GPU|CUDA|cuda"):
        rg.la_gate(torch.zeros(1, 1, 2), torch.zeros(2), torch.zeros(2))
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ImportError):
        rg.la_decode(x, x, x, torch.zeros(1, 2, 3), torch.zeros(1, 2, 64, 64))
    with pytest.raises(ImportError):
        rg.la_norm_gate(x, torch.ones(64))


@pytest.mark.parametrize("missing", ["compiler error", "no torch"])
def test_the_library_is_built_without_the_module(monkeypatch, tmp_path, missing):
    """Where the module cannot be compiled, or torch's headers are missing, librgdr.so is linked all the
    same, and the error is raised."""
    from gated_delta_rule_rgdr_amd import build

    def commands(obj):
        if missing == "no torch":
            raise ImportError("torch")
        return ["false"], ["false"]
    monkeypatch.setattr(build, "SOURCES", ["rgdr_host.cpp"])
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "librgdr.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_la_binding.so"))
    monkeypatch.setattr(build, "binding_cmds", commands)
    with pytest.raises((RuntimeError, ImportError), match="la_binding.cpp|torch"):
        build.build()
    assert (tmp_path / "librgdr.so").exists() and not (tmp_path / "_la_binding.so").exists()
