"""Batches that the header allows beside the usual ones: rows in front of the first request, pages that requests share
or that one lists twice, keys and values in one buffer."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_attention import Batch, check, ints, normal, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = [(8, 2, 64), (8, 2, 128), (6, 1, 256)]


@pytest.mark.parametrize("heads", SIZES)
@pytest.mark.parametrize("new", [1, 8, 70])
def test_rows_in_front_of_the_first_request(vq3, heads, new):  # noqa: F811
    b = Batch(70, [(200, new), (new, new)], *heads, 32, "f16", behind=0)
    T, front = b.starts[-1], 5
    q = torch.full((T + front, *b.q.shape[1:]), float("nan"), dtype=b.q.dtype, device=DEV)
    q[front:] = b.q
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    starts = [s + front for s in b.starts]
    vq3.paged_attention(q, b.k, b.v, b.table, ints(starts), b.kv_len, max_new=new, out=out, lse=lse)
    check(out, lse, q, b.keys, b.values, starts, b.seen, heads[2] ** -0.5, "f16")
    assert (out[:front] == 7.0).all() and (lse[:front] == 7.0).all()
    k, v = (normal(torch.Generator().manual_seed(s), (T + front, heads[1], heads[2]), "f16") for s in (71, 72))
    k[:front] = v[:front] = float("nan")
    out.fill_(7.0)
    vq3.prompt_attention(q, k, v, ints(starts), max_new=new, out=out)
    cut = [slice(starts[r], starts[r + 1]) for r in range(2)]
    check(out, None, q, [k[c] for c in cut], [v[c] for c in cut], starts, [[i + 1 for i in range(new)]] * 2,
          heads[2] ** -0.5, "f16")
    assert (out[:front] == 7.0).all()


@pytest.mark.parametrize("heads", SIZES)
@pytest.mark.parametrize("new", [1, 8, 70])
def test_shared_and_repeated_pages(vq3, heads, new):  # noqa: F811
    # a common prefix of two pages, one page that a request lists twice, keys and values halves of one buffer
    H, Hkv, D = heads
    g = torch.Generator().manual_seed(73)
    page = 64
    pool = normal(g, (9, page, Hkv, 2 * D), "bf16")
    k_pages, v_pages = pool[..., :D], pool[..., D:]
    table = [[4, 1, 7, 2], [4, 1, 0, 8], [6, 3, 6, -1]]
    kv = [230, 128 + 70, 180]
    q = normal(g, (3 * new, H, D), "bf16", 1.5)
    starts = [0, new, 2 * new, 3 * new]
    out = vq3.paged_attention(q, k_pages, v_pages, ints(table), ints(starts), ints(kv), max_new=new)
    keys, values = ([x[[p for p in t if p >= 0]].flatten(0, 1)[:n] for t, n in zip(table, kv)] for x in (k_pages, v_pages))
    check(out, None, q, keys, values, starts, [[n - new + i + 1 for i in range(new)] for n in kv], D**-0.5, "bf16")
