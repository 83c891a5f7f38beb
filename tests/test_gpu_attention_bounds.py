"""The bounds-check build on every kernel path of the attention token mixer: no instrumented global
access is out of range, and the outputs are bit-identical to the normal build's."""

import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(path, lib=None):
    env = dict(os.environ)
    env.pop("VQ3_LIB", None)
    if lib:
        env["VQ3_LIB"] = lib
    r = subprocess.run([sys.executable, "-m", "tests.attention_workloads", str(path)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return np.load(path)


def test_attention_bounds_clean_and_bit_identical(tmp_path):
    from bit_vector_lut_gb300 import build as B
    bc = _run(tmp_path / "bc.npz", B.build(bounds_check=True))
    assert "bounds-check build" in str(bc["version"])
    for f in ("attn", "attn_wide", "kvcache"):
        count, site = bc[f"bounds_{f}"]
        assert count == 0, f"{f}: {count} accesses out of range, first at site {site}"
    ref = _run(tmp_path / "normal.npz")
    names = [n for n in ref.files if n != "version"]
    assert len(names) >= 30
    for n in names:
        assert np.array_equal(bc[n].view(np.uint8), ref[n].view(np.uint8)), f"{n}: the two builds differ"
