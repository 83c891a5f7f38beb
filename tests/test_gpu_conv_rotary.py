"""The short convolution and the rotated append on the GPU against the float64 oracle (oracle/mixers.py),
elementwise; copies exactly. A serving step of both kinds of layers run together is in test_gpu_hybrid.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import mixers as O  # noqa: E402
from tests.test_gpu_delta_batch import DEV, DT, HINTS, f64, ints, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu
HALF = {"f16": 2.0**-11, "bf16": 2.0**-8}  # half a step of the type
TINY = {"f16": 2.0**-25, "bf16": 2.0**-134}
assert HINTS


def long(a):
    return torch.tensor(a, dtype=torch.int64, device=DEV)


# ---------------------------------------------------------------- short convolution

class Conv:
    def __init__(self, seed, new, channels=64, width=4, dtype="f16", bias=False, before=0, behind=2, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        R, T = len(new), before + sum(new) + behind
        self.new, self.dtype = new, dtype
        self.starts = (before + np.concatenate([[0], np.cumsum(new)])).astype(int).tolist()
        self.x = (torch.randn(T, channels, generator=g) * gain).to(DT[dtype])
        self.x[:before] = float("nan")
        self.x[self.starts[-1]:] = float("nan")
        self.w = torch.randn(channels, width, generator=g).to(DT[dtype])
        self.bias = torch.randn(channels, generator=g).to(DT[dtype]) if bias else None
        order = torch.randperm(2 * R + 2, generator=g).tolist()
        self.slot_in, self.slot_out = order[:R], order[R : 2 * R]
        self.states = torch.full((2 * R + 2, width - 1, channels), float("nan"), dtype=DT[dtype])
        self.states[self.slot_in] = (torch.randn(R, width - 1, channels, generator=g) * gain).to(DT[dtype])

    def run(self, vq3, slot_in="own", slot_out="own", **kw):
        pick = lambda s, mine: ints(mine) if isinstance(s, str) else (None if s is None else ints(s))  # noqa: E731
        states = self.states.to(DEV).clone()
        out = torch.full(self.x.shape, 7.0, dtype=DT[self.dtype], device=DEV)
        vq3.short_conv(self.x.to(DEV), self.w.to(DEV), states, ints(self.starts), pick(slot_in, self.slot_in),
                       pick(slot_out, self.slot_out), bias=None if self.bias is None else self.bias.to(DEV), out=out, **kw)
        torch.cuda.synchronize()
        return out, states

    def check(self, out, states, slot_in=None, slot_out=None, silu=True, unit_heads=0, head_dim=0, eps=1e-6):
        slot_in = self.slot_in if slot_in is None else slot_in
        slot_out = self.slot_out if slot_out is None else slot_out
        got, old, now, w = f64(out), f64(self.states), f64(states), f64(self.w)
        bias = None if self.bias is None else f64(self.bias)
        n_slots = len(old)
        for r, n in enumerate(self.new):
            a, b = self.starts[r], self.starts[r + 1]
            s0 = old[slot_in[r]] if 0 <= slot_in[r] < n_slots else np.zeros(old.shape[1:])
            ref, kept, err = O.conv(f64(self.x[a:b]), s0, w, bias, silu, unit_heads, head_dim, eps)
            tol = HALF[self.dtype] * np.abs(ref) + (1 + HALF[self.dtype]) * err + TINY[self.dtype]
            e = np.abs(got[a:b] - ref)
            assert (e <= tol).all(), f"request {r} ({n} tokens): {np.max(e / tol):.2f} of the bound"
            if 0 <= slot_out[r] < n_slots:
                assert np.array_equal(now[slot_out[r]], kept), f"request {r} ({n} tokens): state"
        for s in set(range(n_slots)) - {s for s in slot_out if 0 <= s < n_slots}:
            assert np.array_equal(now[s], old[s], equal_nan=True), f"slot {s} changed"
        assert (got[: self.starts[0]] == 7).all() and (got[self.starts[-1]:] == 7).all()


LENGTHS = [4, 0, 1, 2, 3, 5, 31, 32, 33, 0, 70, 1]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("bias", [False, True])
def test_conv_ragged_batch(vq3, dtype, width, bias):  # noqa: F811
    c = Conv(1, LENGTHS, 72, width, dtype, bias, before=3)
    out, states = c.run(vq3)
    c.check(out, states)


@pytest.mark.parametrize("channels,heads,dim", [(8, 1, 8), (64, 2, 32), (1024, 3, 128), (1096, 4, 256), (2048, 32, 64), (24, 3, 8),
                                                (1032, 8, 128), (4104, 1, 16)])
def test_conv_unit_heads(vq3, channels, heads, dim):  # noqa: F811
    c = Conv(2, [6, 1, 40], channels, 4, "bf16")
    out, states = c.run(vq3, unit_heads=heads, head_dim=dim)
    c.check(out, states, unit_heads=heads, head_dim=dim)


@pytest.mark.parametrize("kw", [dict(silu=False), dict(silu=False, unit_heads=2, head_dim=16), dict(unit_heads=4, head_dim=16, eps=0.5)])
def test_conv_forms(vq3, kw):  # noqa: F811
    c = Conv(3, [9, 2], 64, 4, "f16", True)
    out, states = c.run(vq3, **kw)
    c.check(out, states, **kw)


def test_conv_slots(vq3):  # noqa: F811
    c = Conv(4, [9, 2, 0, 1, 0], 64)
    n = len(c.states)
    ins, outs = [-1, n, -7, c.slot_in[3], c.slot_in[4]], [c.slot_out[0], c.slot_out[1], c.slot_out[2], n, -1]
    out, states = c.run(vq3, ins, outs)
    c.check(out, states, ins, outs)
    out, states = c.run(vq3, None, None)
    c.check(out, states, [-1] * 5, [-1] * 5)
    # in place, short and empty requests among them; one slot read by two
    ins = [c.slot_in[0], c.slot_in[1], c.slot_in[2], c.slot_in[3], c.slot_in[4]]
    out, states = c.run(vq3, ins, ins)
    c.check(out, states, ins, ins)


def test_conv_in_place_over_many_tiles(vq3):  # noqa: F811
    # the slot that a request's first tile reads is the one that takes its state
    c = Conv(5, [700, 3, 900, 1, 1500], 2048, 4, "bf16")
    for _ in range(3):
        out, states = c.run(vq3, c.slot_in, c.slot_in)
        c.check(out, states, c.slot_in, c.slot_in)


def test_conv_large_values(vq3):  # noqa: F811
    # far ends of the sigmoid: no NaN from infinities on the way
    c = Conv(6, [40], 64, 4, "bf16", gain=60.0)
    out, states = c.run(vq3)
    c.check(out, states)


def test_conv_strides(vq3):  # noqa: F811
    c = Conv(7, [33, 2], 64, 4, "f16")
    wide = torch.zeros(len(c.x), 96, dtype=torch.float16, device=DEV)
    x = wide[:, 16:80]
    x.copy_(c.x)
    pool = torch.zeros(len(c.states), 5, 80, dtype=torch.float16, device=DEV)
    states = pool[:, 1:4, 8:72]
    states.copy_(c.states)
    out = torch.full((len(c.x), 88), 7.0, dtype=torch.float16, device=DEV)
    vq3.short_conv(x, c.w.to(DEV), states, ints(c.starts), ints(c.slot_in), ints(c.slot_out), out=out[:, 8:72])
    torch.cuda.synchronize()
    c.check(out[:, 8:72], states)
    assert (out[:, :8] == 7).all() and (out[:, 72:] == 7).all() and (pool[:, 0] == 0).all() and (pool[:, 4] == 0).all()


def test_conv_many_requests_and_repeats(vq3):  # noqa: F811
    c = Conv(8, [i % 3 for i in range(1000)], 16)
    (a, sa), (b, sb) = c.run(vq3), c.run(vq3)
    c.check(a, sa)
    assert torch.equal(a[:-2], b[:-2]) and torch.equal(sa.view(torch.int16), sb.view(torch.int16))


def test_conv_captured_step_serves_other_lengths(vq3):  # noqa: F811
    c = Conv(9, [8, 3, 6], 64, behind=7)
    x, w, states, q_start = c.x.to(DEV), c.w.to(DEV), c.states.to(DEV).clone(), ints(c.starts)
    ins, outs, out = ints(c.slot_in), ints(c.slot_out), torch.full(c.x.shape, 7.0, dtype=torch.float16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vq3.short_conv(x, w, states, q_start, ins, outs, out=out)
    for new in ([8, 3, 6], [1, 8, 8], [0, 5, 0]):
        c.new, c.starts = new, np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
        q_start.copy_(ints(c.starts))
        states.copy_(c.states)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, states)


# ---------------------------------------------------------------- append with rotation

class Rotary:
    """Rows at given positions and slots of a cache of NaN."""

    def __init__(self, seed, positions, heads=3, kv_heads=2, dim=64, rotated=64, page=16, dtype="f16", base=1e4, layout="nhd"):
        g = torch.Generator().manual_seed(seed)
        T = len(positions)
        self.dtype, self.positions, self.page = dtype, positions, page
        self.q, self.k, self.v = (torch.randn(T, h, dim, generator=g).to(DT[dtype]) for h in (heads, kv_heads, kv_heads))
        self.freq = torch.tensor([base ** (-2 * i / rotated) for i in range(rotated // 2)], dtype=torch.float32)
        n_pages = -(-T // page) + 2
        slots = torch.randperm(n_pages * page, generator=g)[:T].tolist()
        self.slots = [s if p >= 0 else -1 for s, p in zip(slots, positions)]
        shape = (n_pages, page, kv_heads, dim) if layout == "nhd" else (n_pages, kv_heads, page, dim)
        pools = [torch.full(shape, 5.0, dtype=DT[dtype], device=DEV) for _ in range(2)]
        self.pages = pools if layout == "nhd" else [p.transpose(1, 2) for p in pools]

    def run(self, vq3, interleaved=False, q="own", q_out=None, **kw):
        q = self.q.to(DEV) if isinstance(q, str) else q
        if q is not None and q_out is None:
            q_out = torch.full(self.q.shape, 7.0, dtype=DT[self.dtype], device=DEV)
        got = vq3.kv_append_rotary(q, self.k.to(DEV), self.v.to(DEV), ints(self.positions), long(self.slots),
                                   self.freq.to(DEV), *self.pages, interleaved=interleaved, q_out=q_out, **kw)
        torch.cuda.synchronize()
        return got

    def check(self, q_out, interleaved=False):
        pos, half = np.array(self.positions), HALF[self.dtype]
        live = pos >= 0
        want_pages = np.full(tuple(self.pages[0].shape), 5.0), np.full(tuple(self.pages[0].shape), 5.0)
        tol_k = np.zeros(want_pages[0].shape)
        ref, tol = O.rotate(f64(self.k), pos, self.freq.numpy(), interleaved)
        n = 2 * len(self.freq)
        tol = np.where(np.arange(ref.shape[-1]) < n, half * np.abs(ref) + (1 + half) * tol + TINY[self.dtype], 0)
        for t, s in enumerate(self.slots):
            if live[t] and 0 <= s < want_pages[0].shape[0] * self.page:
                at = s // self.page, s % self.page
                want_pages[0][at], tol_k[at], want_pages[1][at] = ref[t], tol[t], f64(self.v[t])
        assert (np.abs(f64(self.pages[0]) - want_pages[0]) <= tol_k).all(), "keys"
        assert np.array_equal(f64(self.pages[1]), want_pages[1]), "values"
        if q_out is not None:
            ref, tol = O.rotate(f64(self.q), pos, self.freq.numpy(), interleaved)
            tol = np.where(np.arange(ref.shape[-1]) < n, half * np.abs(ref) + (1 + half) * tol + TINY[self.dtype], 0)
            got = f64(q_out)
            assert (np.abs(got - ref) <= tol)[live].all(), "queries"
            return got, live


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotated", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 96), (256, 256), (256, 64), (256, 80)])
def test_rotary_forms(vq3, dtype, interleaved, dim, rotated):  # noqa: F811
    c = Rotary(1, [0, 1, 2, 77, -1, 4095, 131071, -1, 3], dim=dim, rotated=rotated, dtype=dtype)
    got, live = c.check(c.run(vq3, interleaved), interleaved)
    assert (got[~live] == 7).all()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 1), (24, 4), (7, 7), (2, 3)])
@pytest.mark.parametrize("T", [1, 3, 100, 2500])
def test_rotary_heads_and_tokens(vq3, heads, kv_heads, T):  # noqa: F811
    # 2,500 tokens are above what a CTA a token takes (5 per SM)
    c = Rotary(2, [(i * 37) % 5000 if i % 10 else -1 for i in range(T)], heads, kv_heads, 64, 32, 32, "bf16", layout="hnd")
    got, live = c.check(c.run(vq3))
    assert (got[~live] == 7).all()


def test_rotary_far_positions(vq3):  # noqa: F811
    # the largest positions, and frequencies of any size and sign: angles of 10^9 radians
    c = Rotary(3, [2**31 - 1, 2**30 + 1, 10**9 + 7, 16777217, 2**31 - 2], dim=64, rotated=64)
    c.freq[:6] = torch.tensor([1.0, -1.0, 0.0, 3.14159274, 1e-9, 100.5])
    c.check(c.run(vq3))


def test_rotary_without_queries_and_slots(vq3):  # noqa: F811
    c = Rotary(4, [5, 6, 7, 8])
    assert c.run(vq3, q=None) is None
    c.check(None)
    # a slot behind the cache, a negative one: only the query is turned
    c = Rotary(5, [5, 6, 7, 8])
    c.slots[1], c.slots[2] = c.pages[0].shape[0] * 16, -3
    c.check(c.run(vq3))


def test_rotary_in_place_and_strided(vq3):  # noqa: F811
    c = Rotary(6, list(range(40, 60)), 4, 2, 128, 128, 16, "bf16")
    fused = torch.cat([c.q.flatten(1), c.k.flatten(1), c.v.flatten(1)], 1).to(DEV)
    q, k, v = (x.view(20, -1, 128) for x in fused.split([512, 256, 256], 1))
    k0, v0 = k.clone(), v.clone()
    got = vq3.kv_append_rotary(q, k, v, ints(c.positions), long(c.slots), c.freq.to(DEV), *c.pages, q_out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(k, k0) and torch.equal(v, v0)
    c.check(q)


def test_rotary_without_angle_is_the_append(vq3):  # noqa: F811
    c = Rotary(7, [0] * 50, page=32, dim=128, rotated=128, dtype="bf16")
    q = c.run(vq3)
    other = [torch.full_like(p, 5.0) for p in c.pages]
    vq3.kv_append(c.k.to(DEV), c.v.to(DEV), long(c.slots), *other)
    torch.cuda.synchronize()
    assert torch.equal(q, c.q.to(DEV)) and all(torch.equal(a, b) for a, b in zip(c.pages, other))
