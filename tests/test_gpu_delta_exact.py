"""The delta rule for packed requests on the GPU: outputs as exact as the states, whatever their type and the kernel.
Against the float64 recurrence with the causal bound of oracle/mixers.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import mixers as O  # noqa: E402
from tests.test_gpu_delta_batch import HINTS, Case, f64, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu
FORMS = [(dk, hint) for dk in (64, 128, 256) for hint in HINTS]  # every kernel


def check(c, out, states, what=""):
    """Where the recurrence is finite (and inside the type's range) within the causal bound, elsewhere not finite."""
    got, old, now = f64(out), f64(c.states), f64(states)
    most = 65504.0 if c.dtype == "f16" else 2.0**127
    for r, n in enumerate(c.new):
        a, b = c.starts[r], c.starts[r + 1]
        for h in range(c.heads):
            g = h // (c.heads // c.qk)
            args = [f64(x[a:b, i]) for x, i in ((c.q, g), (c.k, g), (c.v, h), (c.beta, h), (c.alpha, h))]
            with np.errstate(all="ignore"):
                ref, S, tol, tol_s = O.delta_causal(*args, old[c.slot_in[r], h], c.scale, c.dtype)
                e = np.abs(got[a:b, h] - ref)
                fine = np.abs(ref) <= most
                bad = np.argwhere(fine & ~(e <= tol))
                assert len(bad) == 0, (f"{what} request {r} head {h}: {len(bad)} outputs, first (token, column) {bad[0]}: "
                                       f"{got[a:b, h][tuple(bad[0])]} for {ref[tuple(bad[0])]}")
                assert not np.isfinite(got[a:b, h][~fine]).any(), f"{what} request {r} head {h}: finite outputs"
                e, fine = np.abs(now[c.slot_out[r], h] - S), np.isfinite(S).all(axis=0)
                assert (e <= tol_s)[:, fine].all(), f"{what} request {r} head {h}: state off by {e[:, fine].max():.3g}"
                assert not np.isfinite(now[c.slot_out[r], h][~np.isfinite(S)]).any(), f"{what} request {r} head {h}: state"


def axis(c, i, size=1.0):
    x = torch.zeros(c.dk)
    x[i] = size
    return x.to(c.q.dtype)


UP = 1 + 2.0**-8 + 2.0**-12  # 13 bits: just above the middle of two BF16 values; its upper 11 bits are the middle


@pytest.mark.parametrize("dk,hint", FORMS)
def test_bf16_outputs_of_the_state(vq3, dk, hint):  # noqa: F811
    # out = the state's first row, which has to be rounded up
    c = Case(1, [70], 1, 1, dk, 32, "bf16", behind=0)
    c.q[:], c.k[:], c.v[:], c.alpha[:], c.beta[:], c.scale = axis(c, 0), axis(c, 1), 0, 1.0, 0.0, 1.0
    c.states[c.slot_in[0]] = 0
    c.states[c.slot_in[0], 0, 0] = torch.tensor([UP, -UP] * 16)
    out, states = c.run(vq3, hint)
    assert torch.equal(out.cpu().float(), torch.tensor([1.0078125, -1.0078125] * 16).expand(70, 1, 32))
    check(c, out, states)


@pytest.mark.parametrize("dk,hint", FORMS)
def test_bf16_outputs_of_the_strengths(vq3, dk, hint):  # noqa: F811
    # out = b v of the token itself, b to be rounded up
    c = Case(2, [70], 1, 1, dk, 32, "bf16", behind=0)
    c.q[:], c.k[:], c.v[:], c.alpha[:], c.beta[:], c.scale = axis(c, 0), axis(c, 0), 1, 0.0, 0.5 * UP, 1.0
    c.states[c.slot_in[0]] = 0
    out, states = c.run(vq3, hint)
    assert (out == 0.50390625).all()
    check(c, out, states)


@pytest.mark.parametrize("dk,hint", FORMS)
def test_bf16_outputs_of_the_new_values(vq3, dk, hint):  # noqa: F811
    # out = u = v - k . S of the last token, to be rounded up; q does not see S
    c = Case(3, [70], 1, 1, dk, 32, "bf16", behind=0)
    c.q[:], c.k[:], c.v[:], c.alpha[:], c.beta[:], c.scale = axis(c, 1, 2.0), axis(c, 0, 0.5) + axis(c, 1, 0.5), 1, 1.0, 0.0, 1.0
    c.beta[69] = 1.0
    c.states[c.slot_in[0]] = 0
    c.states[c.slot_in[0], 0, 0] = 2 - 2 * UP
    out, states = c.run(vq3, hint)
    assert (out[69] == 1.0078125).all() and (out[:69] == 0).all()
    check(c, out, states)


@pytest.mark.parametrize("dk,hint", FORMS)
def test_keys_of_very_different_entries(vq3, dk, hint):  # noqa: F811
    # BF16 rows whose entries lie 2^-40 apart, against a state that makes up for it
    c = Case(8, [40], 1, 1, dk, 32, "bf16", behind=0)
    s = torch.tensor([2.0 ** -(i % 5 * 8) for i in range(dk)])
    c.k *= s.to(c.k.dtype)
    out, states = c.run(vq3, hint)
    check(c, out, states)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk", [64, 128, 256])
def test_hints_agree(vq3, dtype, dk):  # noqa: F811
    # the kernel that max_new picks changes an output by a rounding that falls the other way at most
    c = Case(9, [75, 30], 1, 2, dk, 48, dtype, behind=0)
    got = [f64(c.run(vq3, hint)[0]) for hint in HINTS]
    step = 2.0**-7 if dtype == "bf16" else 2.0**-10
    for o in got[1:]:
        # two 22-bit results may lie on two sides of a middle: one step of the larger
        assert (np.abs(o - got[0]) <= step * np.maximum(np.abs(o), np.abs(got[0])) + 2.0**-20).all()
        # and seldom do: results within 2^-17 of the columns' sizes, some 2^-13 of the outputs', of a middle
        assert (o != got[0]).mean() <= (2.0**-4 if dtype == "f16" else 2.0**-6)
