"""Argument checks of the attention calls and the paged cache (no GPU): every refusal comes before a
launch, with the documented status; and the oracle's own pins."""

import ctypes
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")
vq3 = pytest.importorskip("bit_vector_lut_gb300.vq3", reason="libvq3.so not built")

from oracle import attention as A  # noqa: E402

P = 0x10000  # an aligned address that is never read
BIG = 1 << 30


def cache(**kw):
    c = dict(kv_heads=4, head_dim=128, page_size=64, n_pages=10, k=P, v=P, k_page=64 * 512, k_token=512, k_head=128,
             v_page=64 * 512, v_token=512, v_head=128)
    c.update(kw)
    return vq3.vq3_kv_cache(**c)


def rows(**kw):
    r = dict(kv_heads=4, head_dim=128, tokens=7, k=P, v=P, k_token=512, k_head=128, v_token=512, v_head=128)
    r.update(kw)
    return vq3.vq3_kv_rows(**r)


def attn(**kw):
    a = dict(type=0, heads=8, tokens=7, requests=2, max_new=4, scale=0.1, q=P, out=2 * P, lse=None, q_start=P,
             q_token=1024, q_head=128, out_token=1024, out_head=128)
    a.update(kw)
    return vq3.vq3_attn(**a)


def paged(a=None, c=None, table=P, max_pages=3, kv_len=P, ws=P, n=BIG):
    return vq3.lib.vq3_paged_attention(ctypes.byref(a or attn()), ctypes.byref(c or cache()), table, max_pages, kv_len,
                                       ws, n, None)


def prompt(a=None, r=None, ws=P, n=BIG):
    return vq3.lib.vq3_prompt_attention(ctypes.byref(a or attn()), ctypes.byref(r or rows()), ws, n, None)


def append(r=None, slots=P, c=None):
    return vq3.lib.vq3_kv_append(ctypes.byref(r or rows()), slots, ctypes.byref(c or cache()), None)


INVALID, ALIGN, UNSUPPORTED, SPACE = -1, -2, -3, -5


@pytest.mark.parametrize("bad,code", [
    (dict(type=2), UNSUPPORTED), (dict(type=-1), UNSUPPORTED), (dict(heads=0), INVALID), (dict(heads=6), INVALID),
    (dict(tokens=-1), INVALID), (dict(requests=-1), INVALID), (dict(requests=8193), UNSUPPORTED),
    (dict(max_new=-1), INVALID), (dict(tokens=1 << 28), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q_start=None), INVALID), (dict(q=P + 8), ALIGN),
    (dict(out=P + 2), ALIGN), (dict(q_start=P + 2), ALIGN), (dict(lse=P + 1), ALIGN), (dict(q_token=0), INVALID),
    (dict(q_head=64), INVALID), (dict(q_head=132), ALIGN), (dict(q_token=-1024), INVALID), (dict(out_head=0), INVALID),
    (dict(out_token=128), INVALID), (dict(out_token=1028), ALIGN), (dict(out=P), INVALID),
    (dict(q_token=1 << 40), INVALID)])
def test_attention_refuses_query_side(bad, code):
    assert paged(attn(**bad)) == code, vq3.lib.vq3_last_error()
    if "tokens" not in bad:
        assert prompt(attn(**bad)) == code, vq3.lib.vq3_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(kv_heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=P + 4), ALIGN), (dict(v=P + 8), ALIGN),
    (dict(k_page=0), INVALID), (dict(v_token=64), INVALID), (dict(v_head=-128), INVALID), (dict(k_token=513), ALIGN)])
def test_attention_and_append_refuse_caches(bad, code):
    assert paged(c=cache(**bad)) == code, vq3.lib.vq3_last_error()
    if "kv_heads" not in bad and "head_dim" not in bad:
        assert append(c=cache(**bad)) == code, vq3.lib.vq3_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(kv_heads=0), INVALID), (dict(head_dim=80), UNSUPPORTED), (dict(tokens=-1), INVALID), (dict(k=None), INVALID),
    (dict(v=P + 8), ALIGN), (dict(k_token=8), INVALID), (dict(v_head=129), ALIGN), (dict(k_head=0), INVALID)])
def test_rows_are_checked(bad, code):
    assert prompt(r=rows(**bad)) == code, vq3.lib.vq3_last_error()
    if "kv_heads" not in bad and "head_dim" not in bad:
        assert append(r=rows(**bad)) == code, vq3.lib.vq3_last_error()


def test_other_refusals():
    assert append(r=rows(head_dim=64)) == INVALID and append(r=rows(kv_heads=2)) == INVALID
    assert append(slots=None) == INVALID and append(slots=P + 4) == ALIGN
    assert append(r=rows(tokens=0, k=None, v=None), slots=None) == 0  # nothing to do
    assert paged(max_pages=0) == INVALID and paged(max_pages=1 << 25) == UNSUPPORTED
    assert paged(table=None) == INVALID and paged(kv_len=None) == INVALID and paged(table=P + 1) == ALIGN
    assert prompt(r=rows(tokens=8)) == INVALID  # rows of k and v are q's
    need = vq3.attention_workspace_bytes(8, 4, 128, 4)
    assert need > 0
    assert paged(n=need - 1) == SPACE and prompt(n=need - 1) == SPACE
    assert paged(ws=None) == INVALID and paged(ws=P + 16) == ALIGN
    # nothing to do: no rows, no requests
    for a in (attn(tokens=0, q=None, out=None), attn(requests=0)):
        assert paged(a, ws=None) == 0
    assert prompt(attn(tokens=0), rows(tokens=0), ws=None) == 0
    lib = vq3.lib
    assert lib.vq3_paged_attention(None, ctypes.byref(cache()), P, 3, P, P, BIG, None) == INVALID
    assert lib.vq3_prompt_attention(ctypes.byref(attn()), None, P, BIG, None) == INVALID
    assert lib.vq3_kv_append(None, P, ctypes.byref(cache()), None) == INVALID


def test_sizes_beyond_the_kernels_counters():
    # tokens * heads of 2^30 and more, and (row block, key tile) pairs beyond 32 bits
    assert paged(attn(tokens=1 << 27, heads=8)) == UNSUPPORTED
    a = attn(tokens=1 << 26, heads=8, requests=8000)
    assert paged(a, max_pages=1 << 23, n=1 << 40) == UNSUPPORTED
    assert "pairs" in vq3.lib.vq3_last_error().decode()


def test_axes_of_one_element_have_any_stride():
    # past every check up to the workspace, which is too small
    a = attn(tokens=1, heads=4, q_token=1, out_token=3)
    assert paged(a, cache(kv_heads=1, n_pages=1, k_head=0, v_head=5, k_page=7, v_page=0), n=1) == SPACE
    assert prompt(a, rows(tokens=1, k_token=0, v_token=3), n=1) == SPACE


def test_workspace_sizes():
    assert vq3.attention_workspace_bytes(8, 3, 128) == 0 and vq3.attention_workspace_bytes(8, 4, 96) == 0
    assert vq3.attention_workspace_bytes(8, 0, 128) == 0 and vq3.attention_workspace_bytes(8, 4, 128, -1) == 0
    for d in (64, 128, 256):
        assert vq3.attention_workspace_bytes(24, 4, d, 0) > 0


def plan_call(**kw):
    d = dict(cached=P, fresh=P, requests=3, page=64, ring=P, ring_size=9, state=P, table=2 * P, max_pages=4,
             max_tokens=20, q_start=P, kv_len=3 * P, slots=P, positions=P, out=5 * P, status=P)
    d.update(kw)
    return vq3.lib.vq3_paged_plan(*d.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(requests=-1), INVALID), (dict(requests=8193), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(ring_size=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_tokens=-1), INVALID), (dict(max_tokens=(1 << 30) + 1), UNSUPPORTED), (dict(cached=None), INVALID), (dict(fresh=None), INVALID), (dict(ring=None), INVALID),
    (dict(state=None), INVALID), (dict(table=None), INVALID), (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID),
    (dict(slots=None), INVALID), (dict(positions=None), INVALID), (dict(out=None), INVALID), (dict(status=None), INVALID),
    (dict(slots=P + 4), ALIGN), (dict(table=P + 2), ALIGN), (dict(out=P), INVALID), (dict(kv_len=P), INVALID),
    (dict(table=P), INVALID)])
def test_plan_refuses(bad, code):
    assert plan_call(**bad) == code, vq3.lib.vq3_last_error()


def test_binding_refuses_before_the_library():
    f, i = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(2, 16, 4, 64, dtype=torch.float16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    bad = [
        lambda: vq3.prompt_attention(f, f, f.bfloat16(), i),            # types
        lambda: vq3.prompt_attention(f, f.float(), f.float(), i),
        lambda: vq3.prompt_attention(f.transpose(0, 2), f, f, i),       # head_dim axis not contiguous
        lambda: vq3.prompt_attention(f, f, f, i.long()),                # lengths not int32
        lambda: vq3.prompt_attention(f, f, f, i, out=f[:2]),            # out unlike q
        lambda: vq3.prompt_attention(f, f, f, i, lse=torch.zeros(3, 5)),
        lambda: vq3.prompt_attention(f, f, f, i, out=f),                # aliases q
        lambda: vq3.paged_attention(f, pages, pages, table[0], i, one),  # table not 2D
        lambda: vq3.paged_attention(f, pages, pages, table, i, i),      # kv_len of another length
        lambda: vq3.paged_attention(f, pages, pages[:1], table, i, one),
        lambda: vq3.paged_attention(f.bfloat16(), pages, pages, table, i, one),
        lambda: vq3.kv_append(f, f, torch.zeros(2, dtype=torch.int64), pages, pages),  # too few slots
        lambda: vq3.kv_append(f, f, torch.zeros(3, dtype=torch.int32), pages, pages),
        lambda: vq3.kv_append(f, f, torch.zeros(3, dtype=torch.int64), pages, pages),  # CPU tensors
        lambda: vq3.paged_plan(i, i, table, i, i, 16, 4),               # lengths of other batches
    ]
    for call in bad:
        with pytest.raises(vq3.Vq3Error):
            call()


def test_bounds_check_variant_compiles(tmp_path):
    from bit_vector_lut_gb300 import build as B
    import os
    r = subprocess.run([B.nvcc(), *B.ARCH, *B.NVCC_FLAGS, "-DVQ3_BOUNDS_CHECK", "-c",
                        os.path.join(B.CSRC, "kvcache.cu"), "-o", str(tmp_path / "x.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]


# ---------------------------------------------------------------- the oracle's pins

def test_oracle_attention_pins():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 2, 8))
    out, lse, mag, _ = A.attend(q, k, v, [1, 0, 5], 0.3)
    # one key: its value; no key: zeros and -inf; all keys: softmax by numpy over explicit scores
    assert np.allclose(out[0, 3], v[0, 1]) and np.allclose(lse[0, 0], 0.3 * q[0, 0] @ k[0, 0])
    assert not out[1].any() and np.isneginf(lse[1]).all()
    s = np.array([0.3 * q[2, 1] @ k[j, 0] for j in range(5)])
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[2, 1], sum(w[j] * v[j, 0] for j in range(5))) and np.isclose(lse[2, 1], np.log(np.exp(s).sum()))
    assert (np.abs(out) <= mag + 1e-15).all()


def test_oracle_plan_pins():
    table = np.array([[4, -1, -1], [7, 2, -1]])
    st, tab, qs, kv, slots, pos, state = A.plan([16, 20], [2, 1], table, [9, 5, 3], 2, 2, 16, 5)
    assert st == 0 and tab.tolist() == [[4, 3, -1], [7, 2, -1]] and qs == [0, 2, 3] and kv == [18, 21]
    assert slots == [48, 49, 36, -1, -1] and pos == [16, 17, 20, -1, -1] and state == (0, 1)
    assert A.plan([16, 20], [2, 1], table, [9, 5, 3], 2, 0, 16, 2)[0] == 5


@pytest.mark.parametrize("scale,code", [(3e38, INVALID), (2.4e38, INVALID), (2.3e38, SPACE), (1e-30, SPACE)])
def test_scale_in_the_kernels_domain(scale, code):
    # scale * log2(e) is what the kernels use: 2.36e38 * 1.4427 is the largest FP32 number
    assert paged(attn(scale=scale), n=1) == code and prompt(attn(scale=scale), n=1) == code


@pytest.mark.parametrize("n", [(1 << 16) + 1, 5 << 25, 1 << 30])
def test_more_heads_than_a_row_counts(n):
    # 5 * 2^25 heads of 32 chunks are 2^30 in 32 bits: another row's size, not an overflow that shows
    c, r = cache(kv_heads=n, head_dim=256, k_head=256, v_head=256), rows(kv_heads=n, head_dim=256, k_head=256, v_head=256)
    c.k_token = c.v_token = r.k_token = r.v_token = 256 * n
    c.k_page = c.v_page = 256 * n
    assert append(r, c=c) == UNSUPPORTED and "kv_heads" in vq3.lib.vq3_last_error().decode()
    assert paged(c=c) == UNSUPPORTED and prompt(r=r) == UNSUPPORTED
