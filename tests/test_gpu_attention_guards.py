"""Starts that do not ascend or lie outside the batch: no row outside is written, no wait gives up, no access of the
bounds-check build leaves its buffer, and what the cut starts still mean is computed."""

import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _run(path, lib=None):
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = {k: v for k, v in os.environ.items() if k != "VQ3_LIB"}
    if lib:
        env["VQ3_LIB"] = lib
    r = subprocess.run([sys.executable, "-m", "tests.attention_guard_workloads", str(path)], cwd=root, env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return np.load(path)


def test_starts_outside_the_batch(tmp_path):
    from bit_vector_lut_gb300 import build as B
    bc = _run(tmp_path / "bc.npz", B.build(bounds_check=True))
    assert "bounds-check build" in str(bc["version"])
    for f in ("attn", "attn_wide", "kvcache"):
        count, site = bc[f"bounds_{f}"]
        assert count == 0, f"{f}: {count} accesses out of range, first at site {site}"
    ref = _run(tmp_path / "normal.npz")
    names = [n for n in ref.files if n != "version"]
    assert len(names) == 3 * 2 * 8 * 2
    for n in names:
        assert np.array_equal(bc[n], ref[n]), f"{n}: the two builds differ"
