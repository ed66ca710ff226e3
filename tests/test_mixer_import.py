"""The binding can be imported on a torch without CUDA; its calls then refuse their arrays."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
from diagonal_state_space_gb300 import _native, api
_native.marshal = lambda: type("Native", (), {"rotary": lambda *a: None})
try:
    api.s5_rotary(torch.zeros(1, 4, 2, 8), torch.arange(4)[None], torch.ones(4, dtype=torch.float64))
except ValueError as e:
    print(e)
"""


def test_import_without_cuda_in_torch():
    out = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert "CUDA tensor" in out.stdout
