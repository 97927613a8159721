"""The operators around the step under the debug build (guarded device indexing) against the release build.

tests/debug_operator_cases.py runs the same seeded calls under each library in
a process of its own: the debug run must end with status OK in every case (no
guarded index fell outside its buffer) and give the release run's bits.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(tmp_path, which):
    out = tmp_path / f"{which}.npz"
    env = dict(os.environ)
    env["MA_LIBRARY"] = which
    env["PYTHONPATH"] = ROOT + os.pathsep + env.get("PYTHONPATH", "")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_operator_cases.py"), str(out)], env=env,
                       capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-3000:]
    return np.load(out)


def test_guards_hold_and_results_match_release_bit_for_bit(tmp_path):
    rel, dbg = _run(tmp_path, "release"), _run(tmp_path, "debug")
    assert int(rel["debug_build"]) == 0 and int(dbg["debug_build"]) == 1
    assert set(rel.files) == set(dbg.files) and len(rel.files) > 60
    for k in sorted(dbg.files):
        if k.endswith("_status"):
            assert int(dbg[k]) == 0 and int(rel[k]) == 0, (k, int(rel[k]), int(dbg[k]))
        elif k != "debug_build":
            assert np.array_equal(rel[k], dbg[k], equal_nan=True), f"{k} differs between the builds"
