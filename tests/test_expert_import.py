"""The package without what the expert-layer operators need of torch and of the
build."""
import os
import subprocess
import sys

import pytest

from dense_gemm_optimisation_fp32_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_import_under_a_torch_without_gpu_support():
    """Such a torch has no streams to ask for; the package imports, and the
    operators refuse its tensors."""
    r = python("""
import torch
del torch._C._cuda_getCurrentRawStream
import dense_gemm_optimisation_fp32_amd as g
g.load_library()
try:
    g.route(torch.zeros(4, 8), 2)
except ValueError as e:
    print("refused:", e)
""")
    assert r.returncode == 0, r.stderr
    assert "refused: logits must be on a GPU" in r.stdout


@pytest.fixture
def stand_in_build(tmp_path, monkeypatch):
    """build() into tmp_path, with a compiler that only writes its output."""
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING_PATH", str(tmp_path / os.path.basename(b.BINDING_PATH)))
    monkeypatch.setattr(b, "_compile_all", lambda jobs, verbose: {log: (0, "") for _, log in jobs})

    def run(cmd, **_):
        headers = [os.path.join(d, "Python.h") for d in cmd if os.path.isabs(d)]
        if b.BINDING_SOURCE in cmd and not any(map(os.path.exists, headers)):
            return subprocess.CompletedProcess(cmd, 1, "", "fatal error: Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    return tmp_path


def test_build_makes_the_binding(stand_in_build, capsys):
    assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and os.path.exists(b.BINDING_PATH)
    assert capsys.readouterr().err == ""


def test_build_of_the_library_needs_no_python_headers(stand_in_build, monkeypatch, capsys):
    """Without them (an installation that only runs Python) the C library is
    built as ever, the binding of another build does not stay, and the reason is
    printed."""
    with open(b.BINDING_PATH, "w") as f:
        f.write("of an earlier build")
    paths = dict(b.sysconfig.get_paths(), include=str(stand_in_build))
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: paths)
    assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.BINDING_PATH)
    assert "Python.h" in capsys.readouterr().err


def test_binding_is_named_for_its_interpreter():
    """Another version of Python does not load it (its types have another layout)."""
    from importlib.machinery import EXTENSION_SUFFIXES

    assert b.BINDING_PATH.endswith("_expert_binding" + EXTENSION_SUFFIXES[0])
    assert sys.implementation.cache_tag.replace("-", "") in b.BINDING_PATH.replace("-", "")
