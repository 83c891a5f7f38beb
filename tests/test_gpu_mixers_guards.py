"""The delta rule for packed requests, the short convolution and the rotated append where memory could suffer: the
bounds-check build on every kernel, starts and slots outside the batch, two calls at once, prompts in a graph, the
status word."""

import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.mixers_workloads import odd_starts  # noqa: E402
from tests.test_gpu_conv_rotary import Conv, Rotary  # noqa: E402
from tests.test_gpu_delta_batch import DEV, DT, Case, f64, ints, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(path, lib=None):
    env = dict(os.environ)
    env.pop("VQ3_LIB", None)
    if lib:
        env["VQ3_LIB"] = lib
    r = subprocess.run([sys.executable, "-m", "tests.mixers_workloads", str(path)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return np.load(path)


def test_bounds_clean_and_bit_identical(tmp_path):
    from bit_vector_lut_gb300 import build as B
    bc = _run(tmp_path / "bc.npz", B.build(bounds_check=True))
    assert "bounds-check build" in str(bc["version"])
    for f in ("delta_batch", "delta_wide", "conv", "rotary"):
        count, site = bc[f"bounds_{f}"]
        assert count == 0, f"{f}: {count} accesses out of range, first at site {site}"
    ref = _run(tmp_path / "normal.npz")
    names = [n for n in ref.files if n != "version"]
    assert len(names) >= 90
    for n in names:
        assert np.array_equal(bc[n].view(np.uint8), ref[n].view(np.uint8)), f"{n}: the two builds differ"


@pytest.mark.parametrize("hint", [0, 1, 8])
def test_starts_and_slots_outside_the_batch(vq3, hint):  # noqa: F811
    # starts are brought into the batch, slots that do not exist mean zeros and nowhere
    c = odd_starts(hint)
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("hint", [0, 1, 8])
def test_descending_starts_are_empty_requests(vq3, hint):  # noqa: F811
    c = Case(43, [0, 6], 1, 2, 64, 32)
    c.q_start = ints([3, 0, 6])
    out, states = c.run(vq3, hint)
    c.check(out, states)


@pytest.mark.parametrize("dk", [64, 128, 256])
def test_requests_of_every_length_in_any_order(vq3, dk):  # noqa: F811
    # single tokens, verify steps and prompts in one call, one request with none, the longest in the middle
    c = Case(44, [1, 7, 6, 0, 130, 5, 64, 1, 65, 2, 8, 33], 2, 4, dk, 48, "bf16")
    for hint in (0, 3, 32):
        out, states = c.run(vq3, hint)
        c.check(out, states, what=str(hint))


def test_more_requests_than_a_block_has_threads(vq3):  # noqa: F811
    c = Case(45, [(i * 7) % 9 for i in range(600)], 1, 1, 64, 16)
    out, states = c.run(vq3)
    c.check(out, states)


def test_two_calls_at_once(vq3):  # noqa: F811
    a, b = Case(46, [300, 40], 2, 4, 128, 128, "bf16"), Case(47, [90, 200, 3], 2, 4, 128, 128, "f16")
    want = [c.run(vq3) for c in (a, b)]
    side = [torch.cuda.Stream() for _ in range(2)]
    dev = []
    for c in (a, b):
        dev.append([x.to(DEV) for x in (c.q, c.k, c.v, c.beta, c.alpha)] + [c.states.to(DEV).clone(), c.q_start, ints(c.slot_in), ints(c.slot_out)])
    outs = [torch.full(c.v.shape, 7.0, dtype=DT[c.dtype], device=DEV) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(3):
        for d, c, s, o in zip(dev, (a, b), side, outs):
            d[5].copy_(c.states)
        torch.cuda.synchronize()
        for d, c, s, o in zip(dev, (a, b), side, outs):
            vq3.delta_rule_batch(*d, scale=c.scale, out=o, stream=s)
        torch.cuda.synchronize()
        for d, o, w in zip(dev, outs, want):
            assert torch.equal(o.view(torch.int16), w[0].view(torch.int16))
            assert torch.equal(d[5].view(torch.int32), w[1].view(torch.int32))


def test_captured_prompts_serve_other_lengths(vq3):  # noqa: F811
    c = Case(48, [200, 3, 97], 1, 2, 128, 80, "f16", behind=4)
    dev = [x.to(DEV) for x in (c.q, c.k, c.v, c.beta, c.alpha)]
    states, q_start, ins, outs = c.states.to(DEV).clone(), c.q_start.clone(), ints(c.slot_in), ints(c.slot_out)
    out = torch.full(c.v.shape, 7.0, dtype=DT["f16"], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vq3.delta_rule_batch(*dev, states, q_start, ins, outs, scale=c.scale, out=out)
    for new in ([200, 3, 97], [1, 250, 40], [0, 0, 300], [2, 2, 2]):
        c.new, c.starts = new, np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
        q_start.copy_(ints(c.starts))
        states.copy_(c.states)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, states, what=str(new))


def test_one_slot_for_many_requests(vq3):  # noqa: F811
    # a shared prefix: every request goes on from one slot, which nobody writes
    c = Case(49, [5, 70, 1, 9], 1, 2, 64, 64)
    ins = [c.slot_in[0]] * 4
    for hint in (0, 8):
        out, states = c.run(vq3, hint, ins)
        c.check(out, states, slot_in=ins)


@pytest.mark.parametrize("hint", [0, 1, 8])
def test_status_word_stays(vq3, hint):  # noqa: F811
    c = Case(50, [130, 2], 1, 2, 128, 32)
    for was in (0, 7):
        status = ints([was])
        out, states = c.run(vq3, hint, status=status)
        c.check(out, states)
        assert status.item() == was


@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("hint", [0, 1, 8])
def test_requests_without_any_row(vq3, dk, hint):  # noqa: F811
    # states go from slot to slot, or become zeros
    c = Case(51, [0, 0, 0], 1, 2, dk, 32, behind=0)
    ins = [c.slot_in[0], -1, c.slot_in[2]]
    out, states = c.run(vq3, hint, ins)
    c.check(out, states, slot_in=ins)


def test_conv_without_any_row(vq3):  # noqa: F811
    import ctypes
    c = Conv(52, [0, 0], 64, 4, behind=0)
    ins = [c.slot_in[0], -1]
    out, states = c.run(vq3, ins)
    c.check(out, states, slot_in=ins)
    # and with null inputs, which the header allows without rows
    states, starts, slots = c.states.to(DEV).clone(), ints([0, 0, 0]), (ints(ins), ints(c.slot_out))
    b = vq3.vq3_batch(0, 2, len(states), starts.data_ptr(), slots[0].data_ptr(), slots[1].data_ptr())
    d = vq3.vq3_conv(0, 64, 4, 1, 0, 0, 1e-6, None, None, None, states.data_ptr(), None, 64, 64, 192, 64)
    assert vq3.lib.vq3_short_conv(ctypes.byref(b), ctypes.byref(d), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    c.check(out, states, slot_in=ins)


@pytest.mark.parametrize("hint", [0, 1, 8])
def test_states_past_32_bits(vq3, hint):  # noqa: F811
    # slots 2^31 floats into the pool, 9 GB
    c = Case(53, [70, 3], 1, 2, 128, 128, "bf16")
    pool = torch.empty(70000, 2, 128, 128, device=DEV)
    ins, outs = [69999, 66000], [65999, 69990]
    for r in range(2):
        pool[ins[r]] = c.states[c.slot_in[r]].to(DEV)
    out = torch.full(c.v.shape, 7.0, dtype=DT["bf16"], device=DEV)
    vq3.delta_rule_batch(*(x.to(DEV) for x in (c.q, c.k, c.v, c.beta, c.alpha)), pool, c.q_start, ints(ins), ints(outs),
                         max_new=hint, scale=c.scale, out=out)
    torch.cuda.synchronize()
    states = c.states.to(DEV).clone()
    for r in range(2):
        states[c.slot_out[r]] = pool[outs[r]]
    c.check(out, states)


def test_rows_past_32_bits(vq3):  # noqa: F811
    # rows of a buffer whose tokens lie 2^26 entries apart, the last ones 2^32 into it
    c = Case(54, [70], 1, 1, 64, 64, "f16", behind=0)
    far = torch.empty(70 << 26, dtype=torch.float16, device=DEV)
    view = [far.as_strided((70, 1, 64), (1 << 26, 64, 1), 64 * i) for i in range(4)]
    for x, y in zip(view, (c.q, c.k, c.v)):
        x.copy_(y.to(DEV))
    view[3].fill_(7.0)
    for hint in (0, 1, 8):
        states = c.states.to(DEV).clone()
        vq3.delta_rule_batch(*view[:3], c.beta.to(DEV), c.alpha.to(DEV), states, c.q_start, ints(c.slot_in), ints(c.slot_out),
                             max_new=hint, scale=c.scale, out=view[3])
        torch.cuda.synchronize()
        c.check(view[3], states)
    w = Conv(55, [70], 64, 4, behind=0)
    view[0].copy_(w.x.to(DEV).unflatten(1, (1, 64)))
    states = w.states.to(DEV).clone()
    vq3.short_conv(view[0][:, 0], w.w.to(DEV), states, ints(w.starts), ints(w.slot_in), ints(w.slot_out), out=view[1][:, 0])
    torch.cuda.synchronize()
    w.check(view[1][:, 0], states)


def test_cache_past_32_bits(vq3):  # noqa: F811
    # pages 2^32 entries into the cache, 9 GB a side
    c = Rotary(56, [5, 77, 4095], 3, 2, 128, 64, 16, "bf16")
    pools = [torch.empty(1 << 20, 16, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    small, slots = c.pages, c.slots
    far = [(1 << 20) * 16 - 1 - s for s in slots]
    c.pages, c.slots = pools, far
    got = c.run(vq3)
    for s, p in zip(small, pools):
        for a, b in zip(slots, far):
            s[a // 16, a % 16] = p[b // 16, b % 16]
    c.pages, c.slots = small, slots
    c.check(got)
