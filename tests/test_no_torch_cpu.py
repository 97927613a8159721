"""The binding in a process where torch cannot be imported: calls on plain device addresses reach the library.

Nothing is launched: the library refuses each call for its shapes or alignment, before it looks for a device."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEAD = """
import sys
sys.modules["torch"] = None  # import torch raises ImportError
import adamw_hybrid_optimizer_muon_b200 as ma
def status(call):
    try:
        call()
    except ma.MAError as e:
        return e.code
    return ma.MA_OK
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", HEAD + code], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.split()


@pytest.mark.parametrize("ptrs,numel,code", [("[4096]", "[-1]", "MA_ERR_SHAPE"), ("[4098]", "[8]", "MA_ERR_ALIGN"),
                                             ("[None]", "[8]", "MA_ERR_NULL"), ("[]", "[]", "MA_OK")])
def test_adamw_on_plain_addresses(ptrs, numel, code):
    out = run(f"p = {ptrs}\n"
              f"print(status(lambda: ma.adamw_step_fused(p, p, p, p, ma.adamw_hparams(), stream=0, gdt=ma.MA_F32, "
              f"numel={numel})) == ma.{code})")
    assert out == ["True"]


def test_muon_on_plain_addresses():
    out = run("print(status(lambda: ma.muon_step_batched([4096], [8192], [12288], ma.muon_hparams(), 0, 0, 0, ma.MA_F32, "
              "(0, -1))) == ma.MA_ERR_SHAPE)")
    assert out == ["True"]


def test_arrays():
    out = run("print(list(ma._ptr_array([4096, None, 1 << 63])) == [4096, None, 1 << 63], list(ma._ptr_array([])))")
    assert out == ["True", "[None]"]
