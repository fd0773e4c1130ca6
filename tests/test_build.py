"""The build's staleness test, and what the package needs of its compiled module
``_binding`` (each case in a process of its own, as a module is imported once);
on the CPU."""
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


def test_build_is_stale_for_another_torch_or_python(monkeypatch, tmp_path):
    from masked_flash_attention_gb300 import build as B
    assert B.torch_version() == torch.__version__
    assert not B.stale()  # (the tests' own start has built)
    with monkeypatch.context() as m:
        m.setattr(B, "torch_version", lambda: "1.0")
        assert B.stale()
    with monkeypatch.context() as m:
        m.setattr(B.sysconfig, "get_config_var", lambda name: "cpython-30")
        assert B.stale()
    with monkeypatch.context() as m:
        m.setattr(B, "BUILT_FOR", str(tmp_path / "none.txt"))
        assert B.stale()
    assert not B.stale()
