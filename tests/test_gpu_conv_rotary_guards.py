"""Starts of the convolution and slots and positions of the rotated append that lie outside the batch or the cache, or
starts that do not ascend: nothing outside is written, no index leaves its buffer, and what is defined is right."""

import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import mixers as O  # noqa: E402
from tests.mixers_guard_workloads import GUARD, SLOTS, STARTS, Conv, Rotary  # noqa: E402
from tests.test_gpu_delta_batch import f64, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HALF, TINY = 2.0**-11, 2.0**-25


@pytest.mark.parametrize("width", [2, 4])
@pytest.mark.parametrize("starts,mean", STARTS)
@pytest.mark.parametrize("slots", SLOTS)
def test_conv_starts_and_slots(vq3, width, starts, mean, slots):  # noqa: F811
    c = Conv(width)
    out, pool = c.run(vq3, starts, *slots)
    assert (out[:GUARD] == 7).all() and (out[-GUARD:] == 7).all()
    assert torch.equal(pool[:GUARD], c.pool[:GUARD]) and torch.equal(pool[-GUARD:], c.pool[-GUARD:])
    if mean is None:
        return
    got, old, now = f64(out[GUARD:-GUARD]), f64(c.pool[GUARD:-GUARD]), f64(pool[GUARD:-GUARD])
    want = old.copy()
    assert (got[: mean[0]] == 7).all() and (got[mean[-1]:] == 7).all()
    for r, (i, o) in enumerate(zip(*slots)):
        a, b = mean[r], mean[r + 1]
        s0 = old[i] if 0 <= i < 6 else np.zeros(old.shape[1:])
        ref, kept, err = O.conv(f64(c.x[GUARD + a : GUARD + b]), s0, f64(c.w), None, True, 2, 16, 1e-6)
        assert (np.abs(got[a:b] - ref) <= HALF * np.abs(ref) + (1 + HALF) * err + TINY).all(), f"request {r}"
        if 0 <= o < 6:
            want[o] = kept
    assert np.array_equal(now, want)


def test_rotary_slots_and_positions(vq3):  # noqa: F811
    c = Rotary()
    q, k, v = c.run(vq3)
    live = [p >= 0 for p in c.positions]
    pos = np.array(c.positions)
    ref, tol = O.rotate(f64(c.q), pos, f64(c.freq), False)
    tol = HALF * np.abs(ref) + (1 + HALF) * tol + TINY
    assert (np.abs(f64(q) - ref) <= tol)[live].all() and (q[[not x for x in live]] == 5).all()
    ref, tol = O.rotate(f64(c.k), pos, f64(c.freq), False)
    tol = HALF * np.abs(ref) + (1 + HALF) * tol + TINY
    kept = {s: t for t, s in enumerate(c.slots) if live[t] and 0 <= s < 32}
    assert len(kept) == 2
    for at in range(len(k) * 16):
        page, s = at // 16, at - 16 * GUARD
        if s in kept:
            t = kept[s]
            assert (np.abs(f64(k[page, at % 16]) - ref[t]) <= tol[t]).all() and torch.equal(v[page, at % 16], c.v[t])
        else:
            assert (k[page, at % 16] == 5).all() and (v[page, at % 16] == 5).all()


def _run(path, lib=None):
    env = dict(os.environ)
    env.pop("VQ3_LIB", None)
    if lib:
        env["VQ3_LIB"] = lib
    r = subprocess.run([sys.executable, "-m", "tests.mixers_guard_workloads", str(path)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return np.load(path)


def test_bounds_clean_and_bit_identical(tmp_path):
    from bit_vector_lut_gb300 import build as B
    bc = _run(tmp_path / "bc.npz", B.build(bounds_check=True))
    assert "bounds-check build" in str(bc["version"])
    for f in ("conv", "rotary"):
        count, site = bc[f"bounds_{f}"]
        assert count == 0, f"{f}: {count} accesses out of range, first at site {site}"
    ref = _run(tmp_path / "normal.npz")
    for n in ref.files:
        if n != "version":
            assert np.array_equal(bc[n].view(np.uint8), ref[n].view(np.uint8)), f"{n}: the two builds differ"
