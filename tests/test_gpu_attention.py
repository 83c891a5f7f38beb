"""The attention calls, the page plan and the append on the GPU against the float64 oracle
(oracle/attention.py), elementwise within the bound that the number formats give; integer outputs
exactly."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention as A  # noqa: E402

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


def ints(a, dtype=torch.int32):
    return torch.tensor(a, dtype=dtype, device=DEV)


def normal(gen, shape, dtype, gain=1.0):
    return (torch.randn(*shape, generator=gen) * gain).to(DT[dtype]).to(DEV)


def check(out, lse, q, keys, values, starts, seen, scale, dtype):
    """out, lse against the oracle; keys[r], values[r]: [L, Hkv, D] of request r; seen[r]: keys per row."""
    got, got_lse = f64(out), None if lse is None else f64(lse)
    D = q.shape[2]
    for r in range(len(starts) - 1):
        a, b = starts[r], starts[r + 1]
        if a == b:
            continue
        k, v = f64(keys[r]), f64(values[r])
        ref, ref_lse, mag, S = A.attend(f64(q[a:b]), k, v, seen[r], scale)
        n = max(1, int(max(seen[r])))
        tol, tol_lse = A.bound(ref, ref_lse, mag, S, n, D, np.abs(v[:n]).max(initial=0), dtype)
        assert np.isfinite(got[a:b]).all(), f"request {r}: non-finite"
        e = np.abs(got[a:b] - ref)
        assert (e <= tol).all(), f"request {r}: {np.max(e / tol):.2f} of the bound, at {np.unravel_index(np.argmax(e / tol), e.shape)}"
        if got_lse is not None:
            empty = np.isneginf(ref_lse)
            assert np.array_equal(np.isneginf(got_lse[a:b]), empty)
            d = np.abs(np.where(empty, 0, got_lse[a:b]) - np.where(empty, 0, ref_lse))
            assert (d <= tol_lse).all(), f"request {r}: lse {np.max(d / tol_lse):.2f} of the bound"


class Batch:
    """A paged batch: (kv_len, new) per request; pages dealt out in random order, everything behind a request's
    keys (the rest of its last page, unused pages) NaN, unused table entries -1."""

    def __init__(self, seed, reqs, heads, kv_heads, dim, page, dtype, layout="nhd", spare=3, behind=2, gain=1.5):
        g = torch.Generator().manual_seed(seed)
        self.reqs, self.dtype, self.page = reqs, dtype, page
        need = [-(-kv // page) for kv, _ in reqs]
        n_pages = sum(need) + spare
        shape = {"nhd": (n_pages, page, kv_heads, dim), "hnd": (n_pages, kv_heads, page, dim),
                 "pad": (n_pages, page, kv_heads, dim + 8)}[layout]

        def pool():
            t = torch.full(shape, float("nan"), dtype=DT[dtype], device=DEV)
            return t.transpose(1, 2) if layout == "hnd" else t[..., :dim]

        self.k, self.v = pool(), pool()
        order = torch.randperm(n_pages, generator=g).tolist()
        width = max(need + [1]) + 1
        table = np.full((len(reqs), width), -1)
        self.keys, self.values = [], []
        for r, (kv, _) in enumerate(reqs):
            k, v = normal(g, (kv, kv_heads, dim), dtype), normal(g, (kv, kv_heads, dim), dtype)
            self.keys.append(k)
            self.values.append(v)
            for i in range(need[r]):
                pg = order.pop()
                table[r, i] = pg
                n = min(page, kv - i * page)
                self.k[pg, :n] = k[i * page : i * page + n]
                self.v[pg, :n] = v[i * page : i * page + n]
        self.starts = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).tolist()
        self.table, self.q_start, self.kv_len = ints(table), ints(self.starts), ints([kv for kv, _ in reqs])
        self.q = normal(g, (self.starts[-1] + behind, heads, dim), dtype, gain)
        self.q[self.starts[-1]:] = float("nan")
        self.seen = [[max(0, kv - n + i + 1) for i in range(n)] for kv, n in reqs]
        self.max_new = max(n for _, n in reqs)

    def run(self, vq3, scale=None, max_new=None, **kw):
        out = torch.full_like(self.q, 7.0)
        lse = torch.full(self.q.shape[:2], 7.0, device=DEV)
        vq3.paged_attention(self.q, self.k, self.v, self.table, self.q_start, self.kv_len,
                            max_new=self.max_new if max_new is None else max_new, scale=scale, out=out, lse=lse, **kw)
        return out, lse

    def check(self, vq3, scale=None, **kw):
        out, lse = self.run(vq3, scale, **kw)
        check(out, lse, self.q, self.keys, self.values, self.starts, self.seen, scale or self.q.shape[2] ** -0.5,
              self.dtype)
        # rows behind the last request stay
        assert (out[self.starts[-1]:] == 7.0).all() and (lse[self.starts[-1]:] == 7.0).all()
        return out, lse


HEADS = [(8, 8, 64), (8, 2, 128), (6, 1, 256), (5, 1, 64), (24, 4, 256), (32, 4, 128)]


# the smallest lengths, tiles' and pages' borders, one request without new tokens
EDGES = [(1, 1), (15, 1), (16, 1), (17, 1), (63, 1), (64, 1), (65, 1), (128, 1), (129, 1), (9, 0), (300, 1)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(vq3, dtype, heads, page):
    Batch(1, EDGES, *heads, page, dtype).check(vq3)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("new", [2, 8])
def test_short_steps(vq3, dtype, heads, new):
    reqs = [(new, new), (40, new), (127 + new, new), (128 + new, new - 1), (500, 1), (90, 0)]
    Batch(2, reqs, *heads, 32, dtype).check(vq3)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("reqs", [[(64, 64)], [(700, 64), (5, 5), (130, 1)], [(129, 129), (257, 128), (1, 1), (300, 43)]],
                         ids=["first", "mixed", "ragged"])
def test_chunks(vq3, dtype, heads, reqs):
    Batch(3, reqs, *heads, 16, dtype).check(vq3)


@pytest.mark.parametrize("reqs", [[(0, 1), (3, 5), (0, 9), (20, 20)], [(0, 40), (100, 300)], [(0, 1)]])
@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 1, 256), (4, 4, 64)])
def test_rows_that_see_nothing(vq3, reqs, heads):
    # fewer keys than new tokens: the first rows see none, their output is zero and lse -inf
    out, lse = Batch(4, reqs, *heads, 16, "f16").check(vq3)
    first = reqs[0][1] - reqs[0][0]
    if first > 0:
        assert (out[:first] == 0).all() and torch.isneginf(lse[:first]).all()


@pytest.mark.parametrize("layout", ["hnd", "pad"])
@pytest.mark.parametrize("new", [1, 8, 70])
def test_cache_layouts(vq3, layout, new):
    Batch(5, [(200, new), (new, new), (333, 1)], 8, 4, 128, 64, "bf16", layout).check(vq3)


@pytest.mark.parametrize("new", [1, 8, 70])
def test_strided_query_and_output(vq3, new):
    b = Batch(6, [(200, new), (new, new)], 6, 2, 128, 64, "f16")
    T = b.q.shape[0]
    wide = torch.full((T, 10, 256), 3.0, dtype=b.q.dtype, device=DEV)
    qv = wide[:, 2:8, 128:]
    qv.copy_(b.q)
    buf = torch.full((6, T, 136), 7.0, dtype=b.q.dtype, device=DEV)
    out = buf.transpose(0, 1)[..., :128]
    vq3.paged_attention(qv, b.k, b.v, b.table, b.q_start, b.kv_len, max_new=b.max_new, out=out)
    check(out, None, b.q, b.keys, b.values, b.starts, b.seen, 128**-0.5, "f16")
    assert (buf[..., 128:] == 7.0).all()
    ref, _ = b.run(vq3)
    assert torch.equal(out[: b.starts[-1]], ref[: b.starts[-1]])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gain,scale", [(1.0, 1e-6), (8.0, 1.0), (40.0, 0.5)])
@pytest.mark.parametrize("new", [1, 40])
def test_flat_and_peaked_scores(vq3, dtype, gain, scale, new):
    # from all keys alike to one key taking everything, with the maximum rising by hundreds along the way
    Batch(7, [(500, new), (77, new)], 8, 2, 128, 32, dtype, gain=gain).check(vq3, scale)


@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 1, 256), (16, 16, 64)])
def test_long_request_split_over_the_gpu(vq3, heads):
    # one request's keys divided between all CTAs, a ragged end
    for new in (1, 8, 100):
        Batch(8, [(20011, new)], *heads, 64, "f16").check(vq3)


@pytest.mark.parametrize("heads", [(16, 2, 128), (12, 2, 256)])
def test_batch_that_memory_cannot_keep_up_with(vq3, heads):
    # more keys and values than L2 holds, read as fast as they arrive: the copies, not the products, set the pace
    reqs = [(9000 + 731 * i, 8) for i in range(14)]
    b = Batch(21, reqs, *heads, 64, "f16")
    out, lse = b.check(vq3)
    for _ in range(20):
        again, lse2 = b.run(vq3)
    n = b.starts[-1]
    assert torch.equal(out[:n], again[:n]) and torch.equal(lse[:n], lse2[:n])


@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 1, 256), (2, 2, 64)])
@pytest.mark.parametrize("requests,new", [(129, 1), (700, 1), (200, 7), (140, 30)])
def test_many_requests(vq3, heads, requests, new):
    # above 128 requests the CTAs' warps share the search for their range; some have no new tokens, some no keys
    rng = np.random.default_rng(requests + new)
    reqs = [(int(kv), int(min(kv + 2, n))) for kv, n in zip(rng.integers(0, 200, requests), rng.integers(0, new + 1, requests))]
    reqs[0], reqs[-1] = (0, 0), (50, 0)
    b = Batch(22, reqs, *heads, 16, "f16")
    b.check(vq3)
    b.check(vq3, max_new=0)


def test_most_requests(vq3):
    b = Batch(23, [(1 + i % 23, 1) for i in range(8192)], 2, 1, 64, 16, "bf16")
    out, lse = b.run(vq3)
    again, lse2 = b.run(vq3, max_new=0)
    pick = [0, 1, 22, 4095, 8190, 8191]
    for r in pick:
        check(out[r : r + 1], lse[r : r + 1], b.q[r : r + 1], [b.keys[r]], [b.values[r]], [0, 1], [b.seen[r]], 64**-0.5, "bf16")
        check(again[r : r + 1], lse2[r : r + 1], b.q[r : r + 1], [b.keys[r]], [b.values[r]], [0, 1], [b.seen[r]],
              64**-0.5, "bf16")


# groups that leave rows of a block over, that cut tokens between blocks, as large as a block and larger
@pytest.mark.parametrize("group", [3, 5, 7, 12, 24, 43, 65, 96, 128, 160])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_groups(vq3, group, dim):
    reqs = [(70, 64), (5, 1), (200, 3), (150, 11)]
    Batch(24, reqs, 2 * group, 2, dim, 32, "bf16").check(vq3)


@pytest.mark.parametrize("group", [3, 6, 48])
def test_prompt_groups(vq3, group):
    g = torch.Generator().manual_seed(25)
    lens = [64, 85, 21, 2, 130]
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    for D in (64, 128, 256):
        q, k, v = (normal(g, (sum(lens), h, D), "f16") for h in (2 * group, 2, 2))
        out = vq3.prompt_attention(q, k, v, ints(starts), max_new=130)
        cut = [slice(starts[r], starts[r + 1]) for r in range(len(lens))]
        check(out, None, q, [k[c] for c in cut], [v[c] for c in cut], starts, [[i + 1 for i in range(n)] for n in lens],
              D**-0.5, "f16")


def test_two_streams_at_once(vq3):
    # calls that overlap on the GPU, each with its own workspace, over one cache
    a, b = (Batch(s, [(9000, n), (300, n)], 8, 2, 128, 64, "f16") for s, n in ((26, 1), (27, 90)))
    want = [x.run(vq3)[0] for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                outs.append((x, vq3.paged_attention(x.q, x.k, x.v, x.table, x.q_start, x.kv_len, max_new=x.max_new)))
    torch.cuda.synchronize()
    for x, o in outs:
        n = x.starts[-1]
        assert torch.equal(o[:n], want[0 if x is a else 1][:n])


def test_graphs_that_share_a_workspace(vq3):
    # two captured calls of different kinds and sizes on one workspace, replayed in turn
    a, b = (Batch(s, [(2000, n), (130, n)], 8, 2, 128, 64, "f16") for s, n in ((28, 1), (29, 70)))
    ws = torch.full((max(vq3.attention_workspace_bytes(8, 2, 128, n) for n in (1, 70)),), 0xCD, dtype=torch.uint8,
                    device=DEV)
    want = [x.run(vq3)[0] for x in (a, b)]
    graphs = []
    for x in (a, b):
        out = torch.empty_like(x.q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            vq3.paged_attention(x.q, x.k, x.v, x.table, x.q_start, x.kv_len, max_new=x.max_new, out=out, ws=ws)
        graphs.append((g, out, x))
    for i in range(9):
        for j in ((0, 1), (1, 0), (0, 0, 1, 1))[i % 3]:
            graphs[j][1].fill_(3.0)
            graphs[j][0].replay()
            n = graphs[j][2].starts[-1]
            assert torch.equal(graphs[j][1][:n], want[j][:n])
            assert vq3.workspace_status(ws) == 0


def test_wrong_max_new_is_only_slower(vq3):
    b = Batch(9, [(300, 70), (20, 1)], 8, 2, 128, 16, "f16")
    for hint in (0, 1, 3, 1000):
        b.check(vq3, max_new=hint)


def test_kv_len_beyond_the_table_and_bad_pages(vq3):
    # kv_len is cut to the table's width, a page outside the cache reads as zeros: no access leaves its buffer
    for new in (1, 40):
        b = Batch(10, [(64, new)], 4, 1, 128, 16, "f16", spare=0)
        table = b.table[:, :4].contiguous()
        out = vq3.paged_attention(b.q, b.k, b.v, table, b.q_start, ints([1000]), max_new=new)
        ref = vq3.paged_attention(b.q, b.k, b.v, table, b.q_start, ints([64]), max_new=new)
        assert torch.equal(out[:new], ref[:new])
        table[0, 1], table[0, 3] = 10**6, -5
        out = vq3.paged_attention(b.q, b.k, b.v, table, b.q_start, b.kv_len, max_new=new)
        k, v = b.keys[0].clone(), b.values[0].clone()
        for x in (k, v):
            x[16:32] = 0
            x[48:64] = 0
        check(out, None, b.q, [k], [v], b.starts, b.seen, 128**-0.5, "f16")


def test_bad_starts_touch_nothing_outside(vq3):
    b = Batch(11, [(64, 4), (64, 4)], 4, 1, 128, 16, "f16", behind=0)
    for starts in ([0, 100, 8], [-5, 4, 8], [0, 8, 4], [8, 8, 8]):
        out = torch.full_like(b.q, 7.0)
        vq3.paged_attention(b.q, b.k, b.v, b.table, ints(starts), b.kv_len, max_new=4, out=out)
        torch.cuda.synchronize()


# a packed batch: the smallest prompts, tile borders, an empty one
PACKED = [[1], [1, 2, 0, 17], [63, 64, 65], [127, 1, 128, 129, 0], [300, 5, 257], [0, 0, 3]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", PACKED, ids=str)
def test_prompts(vq3, dtype, heads, lens):
    g = torch.Generator().manual_seed(12)
    H, Hkv, D = heads
    T = sum(lens)
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    # q, k and v as slices of one fused projection's output, three rows behind the last prompt (NaN)
    fused = normal(g, (T + 3, H + 2 * Hkv, D), dtype, 1.3)
    fused[T:] = float("nan")
    q, k, v = fused[:, :H], fused[:, H : H + Hkv], fused[:, H + Hkv :]
    out = torch.full((T + 3, H, D), 7.0, dtype=DT[dtype], device=DEV)
    lse = torch.full((T + 3, H), 7.0, device=DEV)
    vq3.prompt_attention(q, k, v, ints(starts), max_new=max(lens), out=out, lse=lse)
    cut = [slice(starts[r], starts[r + 1]) for r in range(len(lens))]
    check(out, lse, q, [k[c] for c in cut], [v[c] for c in cut], starts, [[i + 1 for i in range(n)] for n in lens],
          D**-0.5, dtype)
    assert (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()


def test_prompt_with_another_ones_infinities(vq3):
    # a prompt packed behind holds infinities and NaN: those in front are untouched by them
    g = torch.Generator().manual_seed(13)
    lens = [70, 200, 33]
    starts = [0, 70, 270, 303]
    for D in (64, 128, 256):
        q, k, v = (normal(g, (303, h, D), "f16") for h in (4, 2, 2))
        k[270:], v[270:] = float("inf"), float("nan")
        out = vq3.prompt_attention(q, k, v, ints(starts), max_new=200)
        cut = [slice(0, 70), slice(70, 270)]
        check(out, None, q, [k[c] for c in cut], [v[c] for c in cut], starts[:3],
              [[i + 1 for i in range(n)] for n in lens[:2]], D**-0.5, "f16")


def test_same_bits_again_and_on_other_pages(vq3):
    for new in (1, 8, 130):
        b = Batch(14, [(3000, new), (170, new), (140, 1)], 8, 2, 128, 64, "bf16")
        one, lse = b.run(vq3)
        for _ in range(3):
            two, lse2 = b.run(vq3)
            assert torch.equal(one[: b.starts[-1]], two[: b.starts[-1]])
            assert torch.equal(lse, lse2)
        n = b.k.shape[0]
        perm = torch.randperm(n, generator=torch.Generator().manual_seed(1)).to(DEV)
        k, v = torch.empty_like(b.k), torch.empty_like(b.v)
        k[perm], v[perm] = b.k, b.v
        b.k, b.v = k, v
        b.table = torch.where(b.table < 0, b.table, perm[b.table.long().clamp(min=0)].int())
        two, _ = b.run(vq3)
        assert torch.equal(one[: b.starts[-1]], two[: b.starts[-1]])


def test_cache_beyond_32_bit_offsets(vq3):
    # pages whose elements lie past 2^32: 5.2 GB each of keys and values, only the touched pages filled
    n_pages, page = 20000, 256
    need = n_pages * page * 4 * 128 * 2 * 2
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("needs 25 GB of free device memory")
    k = torch.empty(n_pages, page, 4, 128, dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    assert k.numel() > 2**31
    g = torch.Generator().manual_seed(15)
    kv, pages = 600, [n_pages - 1, 3, n_pages - 2]
    rows_k, rows_v = normal(g, (kv, 4, 128), "f16"), normal(g, (kv, 4, 128), "f16")
    slots = torch.tensor([pages[i // page] * page + i % page for i in range(kv)], device=DEV)
    vq3.kv_append(rows_k, rows_v, slots, k, v)
    assert torch.equal(k.view(-1, 4, 128)[slots], rows_k) and torch.equal(v.view(-1, 4, 128)[slots], rows_v)
    for new in (1, 50):
        q = normal(g, (new, 8, 128), "f16")
        out = vq3.paged_attention(q, k, v, ints([pages]), ints([0, new]), ints([kv]), max_new=new)
        check(out, None, q, [rows_k], [rows_v], [0, new], [[kv - new + i + 1 for i in range(new)]], 128**-0.5, "f16")


@pytest.mark.parametrize("new", [1, 8, 70])
def test_other_stream_and_caller_workspace(vq3, new):
    b = Batch(16, [(900, new), (40, new)], 8, 2, 128, 32, "f16")
    ref, _ = b.run(vq3)
    ws = torch.full((vq3.attention_workspace_bytes(8, 2, 128, new),), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(b.q)
    vq3.paged_attention(b.q, b.k, b.v, b.table, b.q_start, b.kv_len, max_new=new, out=out, ws=ws, stream=s)
    free = vq3.paged_attention(b.q, b.k, b.v, b.table, b.q_start, b.kv_len, max_new=new, stream=s)
    s.synchronize()
    n = b.starts[-1]
    assert torch.equal(out[:n], ref[:n]) and torch.equal(free[:n], ref[:n])
    assert vq3.workspace_status(ws) == 0


# ---------------------------------------------------------------- plan and append

def run_plan(vq3, cached, fresh, table, ring, head, count, page, max_tokens):
    t = ints(table)
    p = vq3.paged_plan(ints(cached), ints(fresh), t, ints(ring), ints([head, count]), page, max_tokens)
    return t, p


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("requests,new,page", [(1, 1, 16), (3, 8, 64), (64, 1, 16), (300, 40, 128), (1000, 3, 32), (5, 3000, 256)])
def test_plan(vq3, seed, requests, new, page):
    rng = np.random.default_rng(100 + seed)
    cached = rng.integers(0, 400, requests)
    cached[rng.random(requests) < 0.2] = 0
    fresh = rng.integers(0, new + 1, requests)
    if seed == 1:
        fresh[:] = 0
    if seed == 2:
        cached = (cached // page) * page
    held = -(-cached // page)
    need = -(-(cached + fresh) // page)
    width = int(need.max()) + 1
    free = int((need - held).sum()) + (0 if seed == 3 else 4)
    size = max(1, free + 5)
    ids = rng.permutation(int(held.sum()) + size)
    table = np.full((requests, width), -1)
    at = 0
    for r in range(requests):
        table[r, : held[r]] = ids[at : at + held[r]]
        at += held[r]
    ring, head = ids[at : at + size], int(rng.integers(0, size))
    max_tokens = int(fresh.sum()) + (0 if seed == 4 else 37)
    want = A.plan(cached.tolist(), fresh.tolist(), table, ring.tolist(), head, free, page, max_tokens)
    t, p = run_plan(vq3, cached, fresh, table, ring, head, free, page, max_tokens)
    assert want[0] == 0 and p.status.item() == 0
    assert np.array_equal(t.cpu().numpy(), want[1])
    for got, ref in zip((p.q_start, p.kv_len, p.slots, p.positions), want[2:6]):
        assert got.cpu().tolist() == list(ref)
    assert tuple(p.ring_state.tolist()) == want[6]


@pytest.mark.parametrize("what,status", [("pages", 1), ("width", 2), ("tokens", 4), ("negative", 8), ("head", 8), ("all", 7)])
def test_plan_that_cannot_be_met_takes_nothing(vq3, what, status):
    cached, fresh, table = [20, 0, 5], [50, 40, 0], np.array([[1, 2, -1, -1, -1], [-1] * 5, [3, -1, -1, -1, -1]])
    ring, head, count, max_tokens = [7, 8, 9, 10, 11, 12], 4, 6, 90
    if what in ("pages", "all"):
        count = 4
    if what in ("width", "all"):
        table = table[:, :2]
    if what in ("tokens", "all"):
        max_tokens = 89
    if what == "negative":
        fresh = [50, -1, 0]
    if what == "head":
        head = 6
    t, p = run_plan(vq3, cached, fresh, table, ring, head, count, 16, max_tokens)
    assert p.status.item() == status
    assert np.array_equal(t.cpu().numpy(), table)
    assert p.q_start.tolist() == [0] * 4 and p.kv_len.tolist() == [0] * 3
    assert (p.slots == -1).all() and (p.positions == -1).all() and p.ring_state.tolist() == [head, count]


def test_empty_calls(vq3):
    # no requests, no tokens: nothing written, the ring stays
    table = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    p = vq3.paged_plan(none, none, table, ints([1, 2]), ints([1, 2]), 16, 5)
    assert p.status.item() == 0 and p.q_start.tolist() == [0] and p.ring_state.tolist() == [1, 2]
    assert (p.slots == -1).all() and (p.positions == -1).all()
    p = vq3.paged_plan(ints([3]), ints([0]), ints([[7]]), ints([1]), ints([0, 1]), 16, 0)
    assert p.status.item() == 0 and p.slots.numel() == 0 and p.kv_len.tolist() == [3]
    pages = torch.zeros(2, 16, 2, 64, dtype=torch.float16, device=DEV)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=DEV)
    out = torch.full_like(q, 7.0)
    vq3.paged_attention(q, pages, pages, table, ints([0]), none, out=out)
    vq3.prompt_attention(q, q[:, :2], q[:, 2:], ints([0]), out=out)
    assert (out == 7.0).all()
    assert vq3.prompt_attention(q[:0], q[:0, :2], q[:0, 2:], ints([0, 0])).shape == (0, 4, 64)
    vq3.kv_append(q[:0, :2], q[:0, 2:], torch.empty(0, dtype=torch.int64, device=DEV), pages, pages.clone())


def test_status_word_of_empty_calls(vq3):
    # a workspace that held something else: 0 after a call with nothing to do, as after any other
    pages = torch.zeros(2, 16, 2, 64, dtype=torch.float16, device=DEV)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=DEV)
    none, table = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 4, dtype=torch.int32, device=DEV)
    calls = [lambda ws: vq3.paged_attention(q, pages, pages, table, ints([0]), none, ws=ws),
             lambda ws: vq3.prompt_attention(q, q[:, :2], q[:, 2:], ints([0]), ws=ws),
             lambda ws: vq3.prompt_attention(q[:0], q[:0, :2], q[:0, 2:], ints([0, 0]), ws=ws)]
    for call in calls:
        ws = torch.full((vq3.attention_workspace_bytes(4, 2, 64),), 0xAB, dtype=torch.uint8, device=DEV)
        call(ws)
        assert vq3.workspace_status(ws) == 0


def test_plan_most_requests(vq3):
    R = 8192
    rng = np.random.default_rng(7)
    cached, fresh = rng.integers(0, 64, R), rng.integers(0, 3, R)
    held, need = -(-cached // 16), -(-(cached + fresh) // 16)
    table = np.full((R, 6), -1)
    ids = rng.permutation(60000)
    at = 0
    for r in range(R):
        table[r, : held[r]] = ids[at : at + held[r]]
        at += held[r]
    ring = ids[at:]
    T = int(fresh.sum())
    want = A.plan(cached.tolist(), fresh.tolist(), table, ring.tolist(), 11, len(ring), 16, T)
    t, p = run_plan(vq3, cached, fresh, table, ring, 11, len(ring), 16, T)
    assert p.status.item() == 0 and np.array_equal(t.cpu().numpy(), want[1])
    assert p.slots.tolist() == want[4] and p.q_start.tolist() == want[2]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kv_heads,dim", [(1, 64), (5, 128), (4, 256)])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "pad"])
def test_append(vq3, dtype, kv_heads, dim, layout):
    g = torch.Generator().manual_seed(17)
    T, n_pages, page = 83, 9, 32
    b = Batch(18, [(1, 1)], kv_heads, kv_heads, dim, page, dtype, layout, spare=n_pages - 1)
    b.k.fill_(1.0)
    b.v.fill_(2.0)
    fused = normal(g, (T, 3, kv_heads, dim), dtype)
    k, v = fused[:, 0], fused[:, 2]
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(DEV)
    slots[5], slots[11], slots[40] = -1, n_pages * page, 2**40  # skipped
    want_k, want_v = b.k.clone(), b.v.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < n_pages * page:
            want_k[s // page, s % page] = k[t]
            want_v[s // page, s % page] = v[t]
    vq3.kv_append(k, v, slots, b.k, b.v)
    assert torch.equal(b.k, want_k) and torch.equal(b.v, want_v)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (24, 4, 256), (8, 8, 64)])
def test_serving_run(vq3, dtype, heads):
    """Three requests admitted at different steps: prefill in chunks, verify steps, single tokens. Every step plans its
    pages, appends its rows and attends; all outputs equal the definition over the whole sequences, and the first
    request's match prompt_attention on the whole prompt."""
    H, Hkv, D = heads
    g = torch.Generator().manual_seed(19)
    total = [150, 90, 7]
    q, k, v = ([normal(g, (n, h, D), dtype) for n in total] for h in (H, Hkv, Hkv))
    page, n_pages, width = 16, 20, 12
    k_pages = torch.full((n_pages, page, Hkv, D), float("nan"), dtype=DT[dtype], device=DEV)
    v_pages = torch.full_like(k_pages, float("nan"))
    table = torch.full((3, width), -1, dtype=torch.int32, device=DEV)
    ring = ints(torch.randperm(n_pages, generator=g).tolist())
    state = ints([3, n_pages])
    steps = [[64, 0, 0], [64, 80, 0], [8, 8, 1], [1, 1, 1], [8, 1, 5], [5, 0, 0]]
    done = [0, 0, 0]
    outs = [torch.empty(n, H, D, dtype=DT[dtype], device=DEV) for n in total]
    for fresh in steps:
        pack = lambda x: torch.cat([x[r][done[r] : done[r] + fresh[r]] for r in range(3)])  # noqa: E731
        plan = vq3.paged_plan(ints(done), ints(fresh), table, ring, state, page, sum(fresh) + 3)
        assert plan.status.item() == 0
        state = plan.ring_state
        vq3.kv_append(pack(k), pack(v), plan.slots, k_pages, v_pages)
        o = vq3.paged_attention(pack(q), k_pages, v_pages, table, plan.q_start, plan.kv_len, max_new=max(fresh))
        at = 0
        for r in range(3):
            outs[r][done[r] : done[r] + fresh[r]] = o[at : at + fresh[r]]
            at += fresh[r]
            done[r] += fresh[r]
    assert done == total
    starts = np.concatenate([[0], np.cumsum(total)]).tolist()
    check(torch.cat(outs), None, torch.cat(q), k, v, starts, [[i + 1 for i in range(n)] for n in total], D**-0.5, dtype)
    whole = vq3.prompt_attention(torch.cat(q), torch.cat(k), torch.cat(v), ints(starts), max_new=max(total))
    check(whole, None, torch.cat(q), k, v, starts, [[i + 1 for i in range(n)] for n in total], D**-0.5, dtype)


@pytest.mark.parametrize("new", [1, 8, 40])
def test_captured_step_replays_with_other_lengths(vq3, new):
    """Plan, append and attention captured once; the lengths, rows and ring in device memory change between replays."""
    H, Hkv, D, R, page, width = 8, 2, 128, 3, 16, 40
    g = torch.Generator().manual_seed(20)
    T = R * new
    cached, fresh = ints([0] * R), ints([new] * R)
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    ring, state = ints(list(range(R * width))), ints([0, R * width])
    k_pages = torch.full((R * width, page, Hkv, D), float("nan"), dtype=torch.float16, device=DEV)
    v_pages = torch.full_like(k_pages, float("nan"))
    q, k, v = (normal(g, (T, h, D), "f16") for h in (H, Hkv, Hkv))
    out = torch.empty_like(q)
    ws = torch.empty(vq3.attention_workspace_bytes(H, Hkv, D, new), dtype=torch.uint8, device=DEV)
    plan = vq3.paged_plan(cached, ints([0] * R), table, ring, state, page, T)

    def step():
        vq3.paged_plan(cached, fresh, table, ring, state, page, T, out=plan)
        vq3.kv_append(k, v, plan.slots, k_pages, v_pages)
        vq3.paged_attention(q, k_pages, v_pages, table, plan.q_start, plan.kv_len, max_new=new, out=out, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    have = [[] for _ in range(R)]
    lengths = [0] * R
    for fr in ([new, new, new], [new, 0, 1], [1, new, new], [new] * R):
        fresh.copy_(ints(fr))
        cached.copy_(ints(lengths))
        for x in (q, k, v):
            x.copy_(normal(g, tuple(x.shape), "f16"))
        graph.replay()
        torch.cuda.synchronize()
        assert plan.status.item() == 0
        state.copy_(plan.ring_state)
        starts = np.concatenate([[0], np.cumsum(fr)]).tolist()
        for r in range(R):
            have[r].append((k[starts[r] : starts[r + 1]].clone(), v[starts[r] : starts[r + 1]].clone()))
        keys = [torch.cat([x[0] for x in have[r]]) for r in range(R)]
        values = [torch.cat([x[1] for x in have[r]]) for r in range(R)]
        seen = [[lengths[r] + i + 1 for i in range(fr[r])] for r in range(R)]
        check(out, None, q, keys, values, starts, seen, D**-0.5, "f16")
        lengths = [lengths[r] + fr[r] for r in range(R)]
    assert vq3.workspace_status(ws) == 0
