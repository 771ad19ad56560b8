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


def test_star_import_without_pytorch(fa_lib):
    """The C binding as a whole; what needs PyTorch is found by name."""
    run(f"""
import sys
sys.modules['torch'] = None
from {PKG} import *
assert fa_version() and callable(fa_fwd_tree) and attention_forward
import {PKG} as fa
assert 'attention_tree' in dir(fa) and 'fa_fwd' in dir(fa)
try:
    fa.attention_tree
except ImportError:
    pass
else:
    raise SystemExit('no ImportError')
""")


def test_names_that_are_loaded_when_used(fa_lib):
    run(f"""
import {PKG} as fa
from {PKG} import KVCache, attention_tree, cache_read, cache_write, new_cache, tree_words
from {PKG} import qk_norm_rope, qk_norm_rope_backward
assert fa.attention_tree is attention_tree
try:
    fa.no_such_name
except AttributeError:
    pass
else:
    raise SystemExit('no AttributeError')
""")
