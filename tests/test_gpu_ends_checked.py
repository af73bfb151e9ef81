"""The bounds-checked build's logit adjustments, embedding and gradient clipping against the regular one:
no check may fail, and every output must be the same to the bit (the cases: tests/ends_cases.py)."""

import json
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checked_build_matches_regular_bitwise(tmp_path):
    import newton_schulz_orthogonalized_gb300 as nsm

    import ends_cases
    if not os.path.exists(nsm.LIB_CHECKED):
        pytest.fail(f"{nsm.LIB_CHECKED} is missing: __graft_entry__.build() builds it")
    path = str(tmp_path / "out.npz")
    proc = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "ends_cases.py"), path],
                          env=dict(os.environ, NSM_CHECKED="1"), cwd=ROOT, stdout=subprocess.PIPE,
                          stderr=subprocess.STDOUT, text=True, timeout=900)
    assert proc.returncode == 0, proc.stdout[-4000:]
    with open(os.path.splitext(path)[0] + ".json") as f:
        meta = json.load(f)
    assert meta["checked"] is True
    failed = {name: st for name, st in meta["status"].items() if tuple(st) != (0, 0, 0, 0)}
    assert not failed, failed
    checked = np.load(path)
    regular, status = ends_cases.run(nsm)
    assert all(st == (0, 0, 0, 0) for st in status.values()), status
    assert sorted(regular) == sorted(checked.files)
    for name, want in regular.items():
        got = checked[name]
        assert got.shape == want.shape, name
        assert np.array_equal(got, want), f"{name}: {int((got != want).sum())} bytes differ"
