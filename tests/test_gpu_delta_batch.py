"""The delta rule over packed requests on the GPU against the float64 recurrence, elementwise within the bound of
oracle/mixers.py: every kernel, states in slots, ragged and empty requests, strides, gates at
their limits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import mixers as O  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def vq3():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    from bit_vector_lut_gb300 import vq3 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


class Case:
    """Packed requests of `new` tokens; rows before the first and behind the last are NaN, and so are the slots
    that no request has."""

    def __init__(self, seed, new, qk=1, heads=2, dk=64, dv=64, dtype="f16", before=0, behind=2, spare=2):
        g = torch.Generator().manual_seed(seed)
        R, T = len(new), before + sum(new) + behind
        self.new, self.dtype, self.qk, self.heads, self.dk, self.dv = new, dtype, qk, heads, dk, dv
        self.starts = (before + np.concatenate([[0], np.cumsum(new)])).astype(int).tolist()
        self.q_start = ints(self.starts)

        def unit(h):
            x = torch.randn(T, h, dk, generator=g)
            return (x / x.norm(dim=-1, keepdim=True)).to(DT[dtype])

        self.q, self.k = unit(qk), unit(qk)
        self.v = torch.randn(T, heads, dv, generator=g).to(DT[dtype])
        self.alpha = torch.exp(-torch.rand(T, heads, generator=g) * torch.rand(heads, generator=g))
        self.beta = torch.rand(T, heads, generator=g)
        for x in (self.q, self.k, self.v, self.alpha, self.beta):
            x[:before] = float("nan")
            x[self.starts[-1]:] = float("nan")
        order = torch.randperm(2 * R + spare, generator=g)
        self.slot_in, self.slot_out = order[:R].tolist(), order[R : 2 * R].tolist()
        self.states = torch.full((2 * R + spare, heads, dk, dv), float("nan"))
        self.states[self.slot_in] = torch.randn(R, heads, dk, dv, generator=g)
        self.scale = 0.25

    def run(self, vq3, max_new=0, slot_in="own", slot_out="own", **kw):
        """(out, states) of a call; out starts at 7 everywhere."""
        pick = lambda s, mine: ints(mine) if isinstance(s, str) else (None if s is None else ints(s))  # noqa: E731
        states = self.states.to(DEV).clone()
        kw.setdefault("out", torch.full(self.v.shape, 7.0, dtype=DT[self.dtype], device=DEV))
        out = vq3.delta_rule_batch(*(x.to(DEV) for x in (self.q, self.k, self.v, self.beta, self.alpha)), states,
                                   self.q_start, pick(slot_in, self.slot_in), pick(slot_out, self.slot_out),
                                   max_new=max_new, scale=self.scale, **kw)
        torch.cuda.synchronize()
        return out, states

    def reference(self, r, h, state):
        a, b = self.starts[r], self.starts[r + 1]
        g = h // (self.heads // self.qk)
        args = [f64(x[a:b, i]) for x, i in ((self.q, g), (self.k, g), (self.v, h), (self.beta, h), (self.alpha, h))]
        out, S, info = O.delta(*args, state, self.scale)
        return out, S, *O.delta_bound(out, info, args[2], self.scale, self.dtype, args[0])

    def check(self, out, states, slot_in=None, slot_out=None, what=""):
        """Against the recurrence; states that no request writes and rows outside the requests are as they were."""
        slot_in = self.slot_in if slot_in is None else slot_in
        slot_out = self.slot_out if slot_out is None else slot_out
        got, old, now = f64(out), f64(self.states), f64(states)
        n_slots = len(old)
        for r, n in enumerate(self.new):
            a, b = self.starts[r], self.starts[r + 1]
            for h in range(self.heads):
                s0 = old[slot_in[r], h] if 0 <= slot_in[r] < n_slots else np.zeros((self.dk, self.dv))
                ref, S, tol, tol_s = self.reference(r, h, s0)
                e = np.abs(got[a:b, h] - ref)
                assert (e <= tol).all(), f"{what} request {r} ({n} tokens) head {h}: out {np.max(e / tol):.2f} of the bound"
                if 0 <= slot_out[r] < n_slots:
                    e = np.abs(now[slot_out[r], h] - S)
                    limit = tol_s if n else 0
                    assert (e <= limit).all(), f"{what} request {r} ({n} tokens) head {h}: state off by {e.max():.3g}"
        written = {s for s in slot_out if 0 <= s < n_slots}
        for s in range(n_slots):
            if s not in written:
                assert np.array_equal(now[s], old[s], equal_nan=True), f"slot {s} changed"
        assert (got[: self.starts[0]] == 7).all() and (got[self.starts[-1]:] == 7).all()


HINTS = [0, 1, 8, 16]  # prompts, single tokens, blocks of 8 tokens (twice)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("hint", HINTS)
def test_ragged_batch(vq3, dtype, dk, hint):
    c = Case(1, [5, 0, 1, 70, 32, 33, 8], 2, 4, dk, 48, dtype, before=3)
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 65, 97, 300])
def test_lengths(vq3, n, hint):
    c = Case(n, [n], 1, 1, 128, 64, "f16")
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("dv", [16, 32, 64, 80, 128, 272])
@pytest.mark.parametrize("hint", HINTS)
def test_widths(vq3, dv, hint):
    c = Case(2, [20, 3], 1, 2, 64, dv, "bf16")
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("qk,heads", [(1, 1), (1, 5), (3, 3), (2, 6)])
@pytest.mark.parametrize("hint", HINTS)
def test_shared_heads(vq3, qk, heads, hint):
    c = Case(3, [40, 2], qk, heads, 64, 32, "f16")
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("hint", HINTS)
def test_slots(vq3, hint):
    c = Case(4, [9, 40, 0, 1], 1, 2, 64, 32)
    # from zeros and kept nowhere, by entries outside the pool
    n = len(c.states)
    ins, outs = [-1, n, -7, c.slot_in[3]], [c.slot_out[0], -1, c.slot_out[2], n + 5]
    out, states = c.run(vq3, hint, ins, outs)
    c.check(out, states, ins, outs)
    # no slots at all
    out, states = c.run(vq3, hint, None, None)
    c.check(out, states, [-1] * 4, [-1] * 4)
    # a request goes on in its own slot; one prefix for two requests
    ins = [c.slot_in[0], c.slot_in[1], c.slot_in[2], c.slot_in[1]]
    outs = [c.slot_in[0], c.slot_out[1], c.slot_in[2], c.slot_out[3]]
    out, states = c.run(vq3, hint, ins, outs)
    c.check(out, states, ins, outs)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hint", HINTS)
def test_gates_at_their_limits(vq3, dtype, hint):
    c = Case(5, [75], 1, 5, 64, 32, dtype)
    a, b = c.alpha, c.beta
    a[:, 0], b[:, 0] = 1.0, 1.0                       # nothing forgotten
    a[::7, 1], a[12, 1], a[13, 1] = 0.0, 0.0, 1e-30   # the state starts over
    a[:, 2], b[:, 2] = 1e-20, 0.5                     # nothing kept
    b[:, 3] = 0.0                                     # nothing written
    a[:, 4], b[:, 4] = 0.0, 0.0
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hint", HINTS)
def test_repeated_keys(vq3, dtype, hint):
    # every key alike, nothing forgotten: (I + N)^-1 is bidiagonal where the powers of N reach 10^8
    c = Case(6, [64], 1, 2, 64, 32, dtype)
    c.k[:] = c.k[3].clone()
    c.alpha[:], c.beta[:] = 1.0, 1.0
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("dtype,small,large", [("f16", 2.0**-12, 2.0**12), ("bf16", 2.0**-60, 2.0**60)])
def test_sizes_of_values(vq3, dtype, small, large, hint):
    # columns of very different size, and a state that is far smaller or larger than the values
    c = Case(7, [50, 50], 1, 2, 64, 32, dtype)
    c.v[:, 0] *= small
    c.v[:, 1, ::2] *= large
    c.states[c.slot_in[0]] *= large
    c.states[c.slot_in[1]] *= small
    c.scale = 1.0 if dtype == "bf16" else 2.0**-6  # outputs inside FP16's range
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("hint", HINTS)
def test_short_keys(vq3, hint):
    # keys far from unit length, some of them zero: powers of two in the rows' factors
    c = Case(8, [45], 1, 2, 128, 32, "bf16")
    c.k[:45] *= torch.tensor([2.0 ** -(i % 9 * 5) for i in range(45)])[:, None, None].to(DT["bf16"])
    c.k[::11] = 0
    c.q[:45] *= torch.tensor([2.0 ** (i % 7 * 4) for i in range(45)])[:, None, None].to(DT["bf16"])
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hint", HINTS)
def test_a_bad_head_stays_alone(vq3, dtype, hint):
    # an infinity and a NaN in one head's values and one request's state: the others are none the worse
    c = Case(9, [20, 35], 1, 3, 64, 32, dtype)
    c.v[4, 1, 0], c.v[30, 1, 5] = float("inf"), float("nan")
    c.states[c.slot_in[1], 2, 3, 7] = float("nan")
    out, states = c.run(vq3, hint)
    got, now = f64(out), f64(states)
    for r, h in ((0, 0), (0, 2), (1, 0)):
        ref, S, tol, tol_s = c.reference(r, h, f64(c.states[c.slot_in[r], h]))
        assert (np.abs(got[c.starts[r] : c.starts[r + 1], h] - ref) <= tol).all()
        assert (np.abs(now[c.slot_out[r], h] - S) <= tol_s).all()
    assert not np.isfinite(got[4, 1, 0]) and not np.isfinite(got[30, 1, 5]) and not np.isfinite(got[54, 2, 7])


@pytest.mark.parametrize("hint", HINTS)
def test_strides(vq3, hint):
    # slices of one buffer, gates from a wider one, heads in front of tokens, spaced slots
    c = Case(10, [40, 3, 9], 2, 4, 64, 32, "bf16")
    T = len(c.q)
    rows = torch.cat([c.q.flatten(1), c.k.flatten(1), c.v.flatten(1), torch.zeros(T, 24, dtype=DT["bf16"])], 1).to(DEV)
    q, k, v, _ = rows.split([128, 128, 128, 24], 1)
    gates = torch.cat([c.beta, c.alpha, c.beta], 1).to(DEV)
    pool = torch.zeros(len(c.states), 4 * 64 * 32 + 20, device=DEV)
    states = pool[:, : 4 * 64 * 32].view(-1, 4, 64, 32)
    states.copy_(c.states)
    out = torch.full((4, T, 48), 7.0, dtype=DT["bf16"], device=DEV).transpose(0, 1)[..., :32]
    vq3.delta_rule_batch(q.view(T, 2, 64), k.view(T, 2, 64), v.view(T, 4, 32), gates[:, :4], gates[:, 4:8], states,
                         c.q_start, ints(c.slot_in), ints(c.slot_out), max_new=hint, scale=c.scale, out=out)
    torch.cuda.synchronize()
    c.check(out, states)
    assert (pool[:, 4 * 64 * 32 :] == 0).all()
    assert (out.as_strided((T, 4, 16), out.stride(), out.storage_offset() + 32) == 7).all()


@pytest.mark.parametrize("hint", [0, 1])
def test_more_requests_than_threads(vq3, hint):
    new = [(i * 7) % 4 for i in range(300)]
    c = Case(11, new, 1, 1, 64, 16, "f16")
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("hint", HINTS)
def test_repeats_itself(vq3, hint):
    c = Case(12, [90, 1, 17], 1, 3, 128, 128, "bf16")
    a, b = c.run(vq3, hint), c.run(vq3, hint)
    assert torch.equal(a[0].view(torch.int16)[2:-2], b[0].view(torch.int16)[2:-2])
    assert torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


def test_steps_chain(vq3):
    # a prompt, a verify step whose state is left unwritten, the accepted tokens again, single tokens: one sequence
    c = Case(13, [60], 1, 2, 128, 64, "f16", behind=0)
    dev = [x.to(DEV) for x in (c.q, c.k, c.v, c.beta, c.alpha)]
    states = c.states.to(DEV).clone()
    slot = ints(c.slot_in)
    got = []
    for lo, hi, hint, keep in ((0, 40, 0, True), (40, 48, 8, False), (40, 45, 8, True), (45, 46, 1, True), (46, 60, 16, True)):
        o = vq3.delta_rule_batch(*(x[lo:hi] for x in dev), states, ints([0, hi - lo]), slot, slot if keep else ints([-1]),
                                 max_new=hint, scale=c.scale)
        if keep:
            got.append(o)
    ref, S, tol, tol_s = zip(*(c.reference(0, h, f64(c.states[c.slot_in[0], h])) for h in range(2)))
    out, now = f64(torch.cat(got)), f64(states[c.slot_in[0]])
    for h in range(2):
        assert (np.abs(out[:, h] - ref[h]) <= tol[h]).all() and (np.abs(now[h] - S[h]) <= tol_s[h]).all()


def test_captured_step_serves_other_lengths(vq3):
    c = Case(14, [8, 3, 6], 1, 2, 64, 32, "bf16", behind=4)
    dev = [x.to(DEV) for x in (c.q, c.k, c.v, c.beta, c.alpha)]
    states, q_start = c.states.to(DEV).clone(), c.q_start.clone()
    ins, outs = ints(c.slot_in), ints(c.slot_out)
    out = torch.full(c.v.shape, 7.0, dtype=DT["bf16"], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vq3.delta_rule_batch(*dev, states, q_start, ins, outs, max_new=8, scale=c.scale, out=out)
    for new in ([8, 3, 6], [1, 8, 8], [0, 5, 0]):
        c.new, c.starts = new, np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
        q_start.copy_(ints(c.starts))
        states.copy_(c.states)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, states, what=str(new))


@pytest.mark.parametrize("hint", HINTS)
def test_other_stream(vq3, hint):
    c = Case(15, [30, 2], 1, 2, 64, 32)
    want = c.run(vq3, hint)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    states = c.states.to(DEV).clone()
    dev = [x.to(DEV) for x in (c.q, c.k, c.v, c.beta, c.alpha)]
    ins, outs = ints(c.slot_in), ints(c.slot_out)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    out = vq3.delta_rule_batch(*dev, states, c.q_start, ins, outs, max_new=hint, scale=c.scale, stream=side)
    assert not torch.cuda.current_stream().query()
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out[:32], want[0][:32]) and torch.equal(states.view(torch.int32), want[1].view(torch.int32))


def test_nothing_to_do(vq3):
    c = Case(16, [], 1, 2, 64, 32, behind=3, spare=4)
    out, states = c.run(vq3, 0, None, None)
    assert (out == 7).all() and torch.equal(states.cpu().isnan(), c.states.isnan())
    c = Case(17, [0, 0], 1, 2, 64, 32, behind=0)
    out, states = c.run(vq3, 1)
    c.check(out, states)
