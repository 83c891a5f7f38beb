"""The delta rule for packed requests on the GPU where a chunk's tokens could disturb one another: values of very
different size in one chunk, memories that end in it, infinities and NaN behind good tokens. Against the float64
recurrence with the causal bound of oracle/mixers.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import mixers as O  # noqa: E402
from tests.test_gpu_delta_batch import Case, f64, vq3  # noqa: E402,F401
from tests.test_gpu_delta_exact import FORMS, check  # noqa: E402

pytestmark = pytest.mark.gpu
SIZES = {"f16": (2.0**-10, 6e4), "bf16": (1.0, 2.0**40)}  # of the values, of the large ones


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,hint", FORMS)
def test_a_large_value_behind_small_ones(vq3, dtype, dk, hint):  # noqa: F811
    # one column's, in one token, and a whole row of another head's
    small, large = SIZES[dtype]
    for at in (3, 7, 31, 45, 70, 74):
        c = Case(4, [75, 9], 1, 2, dk, 48, dtype, behind=0)
        c.v *= small
        c.states *= small
        c.v[at, 0, 5] = large
        c.v[at, 1] = large
        out, states = c.run(vq3, hint)
        check(c, out, states, f"at {at}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,hint", FORMS)
@pytest.mark.parametrize("gate", [0.0, 2.0**-60])
def test_small_values_behind_a_large_state(vq3, dtype, dk, hint, gate):  # noqa: F811
    # the memory of a state of 2^40 ends inside a chunk
    for at in (0, 2, 12, 40, 66):
        c = Case(5, [75, 9], 1, 2, dk, 48, dtype, behind=0)
        c.states[c.slot_in[0]] *= 2.0**40
        c.alpha[at, :] = gate
        out, states = c.run(vq3, hint)
        check(c, out, states, f"at {at}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,hint", FORMS)
@pytest.mark.parametrize("where", ["v", "k", "q", "alpha", "beta"])
def test_what_is_not_finite_reaches_no_token_before_it(vq3, dtype, dk, hint, where):  # noqa: F811
    for bad in (float("inf"), float("nan")):
        for at in (7, 68, 74):
            c = Case(6, [75, 9], 1, 2, dk, 48, dtype, behind=0)
            x = getattr(c, where)
            if where == "v":
                x[at, 1, 3] = bad  # one column's
            elif where in "kq":
                x[at, 0, 5] = bad
            else:
                x[at, 1] = bad
            out, states = c.run(vq3, hint)
            check(c, out, states, f"{bad} at {at}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,hint", FORMS)
def test_tokens_before_keys_that_are_too_long(vq3, dtype, dk, hint):  # noqa: F811
    # the last keys, of length 2^8 at full strength, let (I + N)^-1 and the state grow by 2^16 a token
    c = Case(7, [40], 1, 1, dk, 32, dtype, behind=0)
    c.k[37:] = c.k[37].clone() * 2.0**8
    c.beta[37:], c.alpha[37:] = 1.0, 1.0
    out, _ = c.run(vq3, hint)
    ref, _, tol, _ = O.delta_causal(*(f64(x[:, 0]) for x in (c.q, c.k, c.v, c.beta, c.alpha)),
                                    f64(c.states[c.slot_in[0], 0]), c.scale, c.dtype)
    assert (np.abs(f64(out[:37, 0]) - ref[:37]) <= tol[:37]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,hint", FORMS)
def test_a_memory_that_fades_without_new_values(vq3, dtype, dk, hint):  # noqa: F811
    # from zeros, one large value, then none: a small gate leaves little of it, which is all there is
    large, gate = {"f16": (6e4, 2.0**-24), "bf16": (2.0**40, 2.0**-60)}[dtype]
    for first, at in ((0, 1), (0, 5), (3, 7), (9, 12), (3, 45), (40, 44), (65, 70)):
        c = Case(10, [75, 9], 1, 2, dk, 48, dtype, behind=0)
        c.states[c.slot_in] = 0
        c.v[:75] = 0
        c.v[first] = large
        c.alpha[:75] = 1.0
        c.alpha[at] = gate
        c.scale = 1.0 if dtype == "bf16" else 0.125
        out, states = c.run(vq3, hint)
        check(c, out, states, f"{first}, gate at {at}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,hint", FORMS)
def test_mixtures(vq3, dtype, dk, hint):  # noqa: F811
    # values, states and gates of any size and zeros among them, by token, by column and by single entry
    rng = np.random.default_rng(dk + hint)
    up = (lambda n: rng.integers(-14, n)) if dtype == "f16" else (lambda n: rng.integers(-60, 61))
    for seed in range(6):
        c = Case(20 + seed, [int(rng.integers(60, 140)), int(rng.integers(1, 20))], 1, 2, dk, 32, dtype, behind=0)
        T = len(c.v)
        if dtype == "f16":
            c.v.clamp_(-3.9, 3.9)  # (times 2^13 inside the type)
        for _ in range(int(rng.integers(0, 5))):
            t, h, col = int(rng.integers(0, T)), int(rng.integers(0, 2)), int(rng.integers(0, 32))
            where = [c.v[t, h], c.v[t, h, col : col + 1], c.v[t:, h, col], c.v[:t, h], c.v[:, h, col]][int(rng.integers(0, 5))]
            where *= 0.0 if rng.random() < 0.3 else 2.0 ** float(up(14))
        if dtype == "f16":
            c.v.clamp_(-6e4, 6e4)
        for _ in range(int(rng.integers(0, 4))):
            c.alpha[int(rng.integers(0, T)), int(rng.integers(0, 2))] = [0.0, 1.0, 2.0 ** -float(rng.integers(0, 60))][int(rng.integers(0, 3))]
        c.states[c.slot_in[0]] *= [0.0, 1.0, 2.0 ** float(rng.integers(-30, 31))][int(rng.integers(0, 3))]
        out, states = c.run(vq3, hint)
        check(c, out, states, f"seed {seed}")
