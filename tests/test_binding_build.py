"""The extension module is built for one torch and one Python: after either changes it is built again, however new its
file is."""
import os

import torch

from quantized_gemm_moe_b200 import build


def test_module_of_another_torch_is_not_up_to_date(monkeypatch):
    build.build()
    assert build.binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert not build.binding_up_to_date()


def test_module_without_a_record_is_not_up_to_date(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(build, "BINDING_ABI", str(tmp_path / "none"))
    assert not build.binding_up_to_date()


def test_module_is_built_again(monkeypatch, tmp_path):
    """The compiler is called for a module of another torch, and not for one that fits."""
    calls = []

    class Done:
        returncode = 0

    def run(cmd, **kwargs):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return Done()

    build.build()
    module = tmp_path / "_qe_torch.so"
    module.write_bytes(b"")
    os.utime(module, (4e9, 4e9))  # newer than every source
    monkeypatch.setattr(build, "BINDING", str(module))
    monkeypatch.setattr(build, "BINDING_ABI", str(tmp_path / "abi"))
    monkeypatch.setattr(build.subprocess, "run", run)
    (tmp_path / "abi").write_text("torch 1.0.0 cxx11 0 cpython-39\n")
    build.build_binding()
    assert len(calls) == 1 and (tmp_path / "abi").read_text() == build._binding_abi()
    os.utime(module, (4e9, 4e9))
    build.build_binding()
    assert len(calls) == 1
