"""The package without what the expert-layer operators need of torch and of the
build."""
import os
import subprocess
import sys

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
