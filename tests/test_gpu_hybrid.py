"""A small hybrid decoder's token mixers as a server runs them, one captured step for every batch: page plan,
append with rotation and attention in one layer, convolution and delta rule in the other, over prompts, a verify
step that is taken back in part, and single tokens. Against both mixers over each request's whole sequence at
once, in float64."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention as A  # noqa: E402
from oracle import mixers as O  # noqa: E402
from tests.test_gpu_delta_batch import DEV, f64, ints, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu

R, H, HKV, D, PAGE = 3, 4, 2, 64, 16                 # attention
QK, V, DK, DV = 2, 4, 64, 32                         # delta rule
CHANNELS = 2 * QK * DK + V * DV
MOST = 48                                            # tokens of a step
# (new tokens of each request, how many of them stay)
STEPS = [([20, 3, 0], [20, 3, 0]), ([1, 8, 30], [1, 2, 30]), ([1, 6, 1], [1, 6, 1]), ([8, 0, 8], [5, 0, 8]), ([3, 1, 1], [3, 1, 1])]


def inputs(seed, total):
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=g).half()  # noqa: E731
    return [{"q": f(n, H, D), "k": f(n, HKV, D), "v": f(n, HKV, D), "x": f(n, CHANNELS),
             "alpha": torch.exp(-torch.rand(n, V, generator=g)), "beta": torch.rand(n, V, generator=g)} for n in total]


def reference(seq, freq, w):
    """Both mixers over one request's sequence, as FP16 tensors pass between the calls."""
    n = len(seq["x"])
    pos = np.arange(n)
    turned = [torch.from_numpy(O.rotate(f64(seq[x]), pos, freq.numpy(), False)[0]).half() for x in ("q", "k")]
    att, _, mag, _ = A.attend(f64(turned[0]), f64(turned[1]), f64(seq["v"]), list(range(1, n + 1)), D**-0.5)
    y, _, _ = O.conv(f64(seq["x"]), np.zeros((3, CHANNELS)), f64(w), None, True, 2 * QK, DK, 1e-6)
    y = f64(torch.from_numpy(y).half())
    q, k, v = np.split(y, [QK * DK, 2 * QK * DK], 1)
    q, k, v = q.reshape(n, QK, DK), k.reshape(n, QK, DK), v.reshape(n, V, DV)
    out = np.empty((n, V, DV))
    size = np.empty((n, V, DV))
    for h in range(V):
        out[:, h], _, info = O.delta(q[:, h // 2], k[:, h // 2], v[:, h], f64(seq["beta"][:, h]), f64(seq["alpha"][:, h]),
                                     np.zeros((DK, DV)), DK**-0.5)
        size[:, h] = DK**-0.5 * (info["reach"] + info["near"])
    return att, mag, out, size


@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps(vq3, captured):  # noqa: F811
    total = [sum(kept[r] for _, kept in STEPS) for r in range(R)]
    seqs = inputs(1, [t + 8 for t in total])
    freq = torch.tensor([1e4 ** (-i / 16) for i in range(16)], dtype=torch.float32)
    w = torch.randn(CHANNELS, 4, generator=torch.Generator().manual_seed(2)).half()
    dev_freq, dev_w = freq.to(DEV), w.to(DEV)
    pages = [torch.full((24, PAGE, HKV, D), float("nan"), dtype=torch.float16, device=DEV) for _ in range(2)]
    table, ring, ring_state = ints([[-1] * 6] * R), torch.randperm(24).to(torch.int32).to(DEV), ints([0, 24])
    conv_pool = torch.zeros(R + 1, 3, CHANNELS, dtype=torch.float16, device=DEV)
    pool = torch.zeros(R + 1, V, DK, DV, device=DEV)
    slot = ints([2, 0, 3])
    buf = {x: torch.zeros(MOST, *seqs[0][x].shape[1:], dtype=seqs[0][x].dtype, device=DEV) for x in seqs[0]}
    cached, fresh, slot_out = ints([0] * R), ints([0] * R), slot.clone()
    plan = vq3.paged_plan(cached, fresh, table, ring, ring_state, PAGE, MOST)
    got = {"att": torch.zeros(MOST, H, D, dtype=torch.float16, device=DEV),
           "delta": torch.zeros(MOST, V, DV, dtype=torch.float16, device=DEV)}
    q_turned = torch.zeros_like(buf["q"])

    def attend():
        vq3.paged_plan(cached, fresh, table, ring, ring_state, PAGE, MOST, out=plan)
        vq3.kv_append_rotary(buf["q"], buf["k"], buf["v"], plan.positions, plan.slots, dev_freq, *pages, q_out=q_turned)
        vq3.paged_attention(q_turned, *pages, table, plan.q_start, plan.kv_len, out=got["att"])

    def mix():
        y = vq3.short_conv(buf["x"], dev_w, conv_pool, plan.q_start, slot, slot_out, unit_heads=2 * QK, head_dim=DK)
        q, k, v = y.split([QK * DK, QK * DK, V * DV], 1)
        vq3.delta_rule_batch(q.view(MOST, QK, DK), k.view(MOST, QK, DK), v.view(MOST, V, DV), buf["beta"], buf["alpha"],
                             pool, plan.q_start, slot, slot_out, scale=DK**-0.5, out=got["delta"])

    calls = {"attend": attend, "mix": mix}
    if captured:
        for name, call in list(calls.items()):
            call()  # no tokens: nothing happens but the first call's work
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            calls[name] = graph.replay

    outs = {"att": [[] for _ in range(R)], "delta": [[] for _ in range(R)]}
    done = [0] * R

    def load(new):
        start = np.concatenate([[0], np.cumsum(new)]).tolist()
        for x, b in buf.items():
            b.fill_(float("nan"))
            for r in range(R):
                b[start[r] : start[r + 1]] = seqs[r][x][done[r] : done[r] + new[r]].to(DEV)
        cached.copy_(ints(done))
        fresh.copy_(ints(new))
        return start

    for new, kept in STEPS:
        start = load(new)
        slot_out.copy_(slot if new == kept else ints([-1] * R))  # a verify step leaves the states alone
        calls["attend"]()
        calls["mix"]()
        torch.cuda.synchronize()
        assert plan.status.item() == 0
        for name, o in outs.items():
            for r in range(R):
                o[r].append(got[name][start[r] : start[r] + kept[r]].clone())
        # pages beyond the kept tokens go back to the ring
        held = [-(-(d + n) // PAGE) for d, n in zip(done, new)]
        need = [-(-(d + n) // PAGE) for d, n in zip(done, kept)]
        head, count = plan.ring_state.tolist()
        for r in range(R):
            for p in range(need[r], held[r]):
                ring[(head + count) % 24] = table[r, p]
                table[r, p] = -1
                count += 1
        ring_state.copy_(ints([head, count]))
        if new != kept:  # the accepted tokens again, for the states
            start = load(kept)
            vq3.paged_plan(cached, fresh, table.clone(), ring, ring_state, PAGE, MOST, out=plan._replace(ring_state=ints([0, 0])))
            slot_out.copy_(slot)
            calls["mix"]()
            torch.cuda.synchronize()
        done = [d + n for d, n in zip(done, kept)]

    for r in range(R):
        seq = {x: t[: total[r]] for x, t in seqs[r].items()}
        att, mag, mixed, size = reference(seq, freq, w)
        # FP16 between the calls, each value of one half step 2^-11: rotated queries and keys turn into scores off by up
        # to 2 * 2^-11 |q| |k| / sqrt(D) (some 2^-7 here), probabilities by as much of themselves on either side
        score = 2 * 2.0**-11 * max(np.linalg.norm(f64(seq["q"]), axis=2).max() * np.linalg.norm(f64(seq["k"]), axis=2).max(), 1) / 8
        e = np.abs(f64(torch.cat(outs["att"][r])) - att)
        assert (e <= (2 * score + 2.0**-9) * mag + 2.0**-20).all(), f"attention of request {r}"
        # a rounding of the convolution's output that falls the other way moves q, k and v by 2^-10 of themselves
        e = np.abs(f64(torch.cat(outs["delta"][r])) - mixed)
        assert (e <= 2.0**-11 * np.abs(mixed) + 2.0**-10 * 4 * size + 2.0**-20).all(), f"delta rule of request {r}"
