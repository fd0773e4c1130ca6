"""What the package needs of its compiled module ``_binding``, on the CPU: each
case in a process of its own, as a module is imported once."""
import os
import subprocess
import sys

import pytest
import torch

import masked_flash_attention_gb300 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = '''
import sys, types
name = "masked_flash_attention_gb300._binding"
{setup}
import torch
import masked_flash_attention_gb300 as fa
q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
assert fa.fa_fwd_plan(q, q, q)[0] == 0           # the calls through ctypes need no module
assert fa.fa_rope_inv_freq(64)[0].numel() == 32
f = torch.ones(8, dtype=torch.float64)
i = torch.ones(1, dtype=torch.int32)
for call in (lambda: fa.fa_rope(q, inv_freq=f), lambda: fa.fa_kvcache_append(q, q, q, q, i),
             lambda: fa.fa_fwd_chunk(q, q, q, i, max_seqlen_k=4), lambda: fa.fa_fwd_chunk_plan(q, q, q, i, max_seqlen_k=4)):
    try:
        call()
    except ImportError as e:
        assert "build()" in str(e) and "{says}" in str(e), e
    else:
        raise AssertionError("no ImportError")
'''


@pytest.mark.parametrize("setup,says", [
    ("sys.modules[name] = None", "does not load"),
    ("m = sys.modules[name] = types.ModuleType(name); m.ABI_VERSION, m.TORCH_VERSION = 8, '1.0'", "torch 1.0"),
    ("m = sys.modules[name] = types.ModuleType(name); import torch; m.ABI_VERSION, m.TORCH_VERSION = 0, torch.__version__", "ABI 0"),
])
def test_package_without_its_compiled_module(setup, says):
    r = subprocess.run([sys.executable, "-c", WITHOUT.format(setup=setup, says=says)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_compiled_module_is_of_this_torch():
    assert fa._ops._binding.TORCH_VERSION == torch.__version__
