"""Attention calls on a stream of the caller's while the current stream still works on memory that was just freed
there: the calls' own buffers are none of that memory."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_attention import Batch, ints, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu
DEV = "cuda"
BUSY = 400_000_000  # cycles that the current stream is kept busy: some 0.2 s


def occupy(sizes):
    """Freed blocks of these sizes (bytes) that the current stream fills with 0xFF once it gets to it."""
    torch.cuda.synchronize()
    blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda._sleep(BUSY)
    for b in blocks:
        b.fill_(255)


@pytest.mark.parametrize("new", [1, 8, 70])
def test_attention_beside_a_busy_stream(vq3, new):  # noqa: F811
    b = Batch(40, [(3000, new), (170, new)], 8, 2, 128, 64, "f16", behind=0)
    want, _ = b.run(vq3)
    side = torch.cuda.Stream()
    sizes = [want.numel() * 2, vq3.attention_workspace_bytes(8, 2, 128, new)]
    for _ in range(3):
        occupy(sizes)
        out = vq3.paged_attention(b.q, b.k, b.v, b.table, b.q_start, b.kv_len, max_new=new, stream=side)
        assert not torch.cuda.current_stream().query()  # the current stream is still at it
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_prompt_beside_a_busy_stream(vq3):  # noqa: F811
    g = torch.Generator().manual_seed(41)
    q, k, v = (torch.randn(300, h, 128, generator=g).half().to(DEV) for h in (8, 2, 2))
    starts = ints([0, 100, 300])
    want = vq3.prompt_attention(q, k, v, starts, max_new=200)
    side = torch.cuda.Stream()
    occupy([want.numel() * 2, vq3.attention_workspace_bytes(8, 2, 128, 200)])
    out = vq3.prompt_attention(q, k, v, starts, max_new=200, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_plan_beside_a_busy_stream(vq3):  # noqa: F811
    args = [ints(x) for x in ([20, 0, 16], [30, 40, 1])]
    table, ring, state = ints([[3, 9, -1, -1], [-1] * 4, [5, -1, -1, -1]]), ints([1, 2, 4, 6, 7, 8, 0]), ints([5, 7])
    want = vq3.paged_plan(*args, table.clone(), ring, state, 16, 80)
    tables = [table.clone() for _ in range(3)]
    side = torch.cuda.Stream()
    for t in tables:
        occupy([4 * x.numel() for x in want] + [8 * 80])
        p = vq3.paged_plan(*args, t, ring, state, 16, 80, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(p, want):
            assert torch.equal(a, b)


def test_result_used_on_the_current_stream_after_a_wait(vq3):  # noqa: F811
    # handed back, read on the current stream behind its other work and freed: the next call's result is elsewhere
    b = Batch(42, [(900, 8)], 8, 2, 128, 64, "f16", behind=0)
    want, _ = b.run(vq3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sums = []
    for i in range(4):
        out = vq3.paged_attention(b.q, b.k, b.v, b.table, b.q_start, b.kv_len, max_new=8, stream=side,
                                  scale=128**-0.5 if i % 2 == 0 else 1e-3)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(BUSY // 8)
        sums.append(out.clone())
        del out
    torch.cuda.synchronize()
    assert torch.equal(sums[0], want) and torch.equal(sums[2], want) and torch.equal(sums[1], sums[3])
    assert not np.array_equal(sums[1].cpu().numpy(), want.cpu().numpy())
