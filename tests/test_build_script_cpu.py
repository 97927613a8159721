"""The build as a module and as a plain script. (The tree is built: nothing is compiled here.)"""
import os
import subprocess
import sys

import pytest

from adamw_hybrid_optimizer_muon_b200 import build as b


@pytest.mark.parametrize("args", [["-m", "adamw_hybrid_optimizer_muon_b200.build"], [b.__file__]])
def test_build_runs(args):
    r = subprocess.run([sys.executable, *args], capture_output=True, text=True, cwd=b.ROOT, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert os.path.samefile(r.stdout.split()[-1], b.LIB)
