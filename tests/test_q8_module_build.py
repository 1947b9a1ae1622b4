"""The binding's native module belongs to one torch: another gets none."""

import os
import shutil

import pytest

from dense_fp32_gemm_row_gb300 import build as gbuild
from dense_fp32_gemm_row_gb300 import q8

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()


def test_a_module_for_another_torch_is_not_used(monkeypatch):
    monkeypatch.setattr(q8, "_native", None)
    q8._load_torch()
    assert q8._native is not None
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    q8._load_torch()
    assert q8._native is None
    monkeypatch.undo()
    q8._load_torch()


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The build's files in a folder of the test's, with a module there that some build left."""
    module = tmp_path / "_tensors.so"
    module.write_bytes(b"an earlier module")
    monkeypatch.setattr(gbuild, "TENSORS", str(module))
    monkeypatch.setattr(gbuild, "TENSORS_FOR", str(tmp_path / "tensors.txt"))
    return module


def test_a_failed_build_leaves_no_module_behind(monkeypatch, tmp_path, elsewhere, capfd):
    broken = tmp_path / "broken.cpp"
    broken.write_text("#error this torch has none of it\n")
    monkeypatch.setattr(gbuild, "TENSORS_SRC", str(broken))
    gbuild._build_tensors(True)
    assert not elsewhere.exists() and "not built" in capfd.readouterr().err


def test_a_missing_compiler_is_reported(monkeypatch, elsewhere, capfd):
    monkeypatch.setattr(gbuild, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setenv("PATH", "/nowhere")
    gbuild._build_tensors(True)
    assert not elsewhere.exists() and "not built" in capfd.readouterr().err


def test_another_version_is_another_module(monkeypatch, elsewhere):
    """Whatever the files' times: packages are unpacked with the times they were made at."""
    compiled = []

    def run(cmd, **_):
        compiled.append([a for a in cmd if "TENSORS_TORCH" in a])
        shutil.copy(gbuild.__file__, cmd[cmd.index("-o") + 1])
        return type("Done", (), {"returncode": 0, "stderr": ""})()

    monkeypatch.setattr(gbuild.subprocess, "run", run)
    version = gbuild._torch_version(os.path.dirname(torch.__file__))
    assert version == str(torch.__version__)
    gbuild._build_tensors(False)
    gbuild._build_tensors(False)
    assert compiled == [[f'-DTENSORS_TORCH="{version}"']]  # the second had nothing to do
    monkeypatch.setattr(gbuild, "_torch_version", lambda _: "2.0.1")
    gbuild._build_tensors(False)
    assert compiled[1:] == [['-DTENSORS_TORCH="2.0.1"']]
