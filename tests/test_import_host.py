"""What importing the package needs: the C binding no PyTorch, flash attention no tensor_calls.so."""
import os
import subprocess
import sys

from conftest import ROOT

PKG = "exact_tiled_attention_26_gb300"


def run(code):
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert p.returncode == 0, p.stderr


def test_flash_attention_without_the_native_calls(fa_lib):
    run(f"""
import sys
sys.modules['{PKG}.tensor_calls'] = None  # as where it is missing or built for another PyTorch
from {PKG}.autograd import flash_attention, qk_norm_rope
import torch
x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
try:
    qk_norm_rope(x, x)
except ImportError as e:
    assert 'tensor_calls.so' in str(e)
else:
    raise SystemExit('no ImportError')
""")
