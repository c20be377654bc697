"""The training-side operators on the bounds-checked build: no index check fails, and every
output equals the release build's bit for bit."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_bounds_checked_operators_are_silent_and_bitwise_equal(tmp_path):
    from tests import operators_battery
    path = tmp_path / "operators.npz"
    pr = subprocess.run([sys.executable, "-m", "tests.operators_battery", str(path)], cwd=ROOT,
                        env=dict(os.environ, DPOPT_LIB_VARIANT="bounds"), capture_output=True,
                        text=True, timeout=300)
    assert pr.returncode == 0, pr.stdout + pr.stderr
    got = np.load(path)
    assert str(got["__version__"]).endswith("+bounds")
    bad = [(n, int(s)) for n, s in zip(got["__names__"], got["__status__"]) if s != 0]
    assert not bad, bad
    want, status = operators_battery.run()
    assert all(s == 0 for _, s in status), status
    assert sorted(want) == sorted(k for k in got.files if not k.startswith("__"))
    for k, v in want.items():
        assert got[k].tobytes() == v.tobytes(), k
