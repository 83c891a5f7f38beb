"""The largest batches that the attention calls take, and what their arguments do not change (no GPU: every call
here ends at its workspace's size or before)."""

import pytest

torch = pytest.importorskip("torch")
vq3 = pytest.importorskip("bit_vector_lut_gb300.vq3", reason="libvq3.so not built")

from tests.test_attention_buffers_cpu import Tensor, run_paged, world  # noqa: E402,F401
from tests.test_attention_cpu import SPACE, UNSUPPORTED, attn, cache, paged, prompt, rows  # noqa: E402


def long_prompt(tokens, heads, kv_heads, dim, max_new, n):
    a = attn(tokens=tokens, requests=1, heads=heads, max_new=max_new, q_token=heads * dim, q_head=dim,
             out_token=heads * dim, out_head=dim)
    r = rows(tokens=tokens, kv_heads=kv_heads, head_dim=dim, k_token=kv_heads * dim, v_token=kv_heads * dim, k_head=dim,
             v_head=dim)
    return prompt(a, r, n=n)


@pytest.mark.parametrize("tokens,heads,kv_heads,dim", [(1 << 18, 32, 8, 128), (1 << 20, 32, 8, 128), (1 << 20, 32, 32, 64),
                                                       (1 << 20, 32, 8, 256)])
def test_max_new_does_not_decide_what_is_taken(tokens, heads, kv_heads, dim):
    need = vq3.attention_workspace_bytes(heads, kv_heads, dim, 0)
    for max_new in (0, 1, 2, tokens):
        mine = vq3.attention_workspace_bytes(heads, kv_heads, dim, max_new)
        assert 0 < mine <= need
        # refused for its workspace alone, by one byte
        assert long_prompt(tokens, heads, kv_heads, dim, max_new, need - 1) == SPACE, (max_new, vq3.lib.vq3_last_error())


def test_what_the_workspace_has_to_hold_is_said():
    mine, need = (vq3.attention_workspace_bytes(32, 8, 128, n) for n in (1, 0))
    assert mine < need and long_prompt(1 << 18, 32, 8, 128, 1, mine) == SPACE
    assert f"{need} bytes, those of max_new 0" in vq3.lib.vq3_last_error().decode()


def test_paged_batches():
    # a table of 2^20 keys a request: 65,536 rows of 32 heads are too many blocks of 8, not of 256
    a = attn(tokens=1 << 16, requests=1, heads=32, max_new=1, q_token=4096, out_token=4096)
    c = cache(kv_heads=8, page_size=256, k_token=1024, v_token=1024, k_page=256 * 1024, v_page=256 * 1024)
    need = vq3.attention_workspace_bytes(32, 8, 128, 0)
    assert paged(a, c, max_pages=4096, n=need - 1) == SPACE


def test_groups_above_a_block_have_one_kernel():
    for max_new in (0, 1, 1 << 20):
        assert long_prompt(1 << 20, 160, 1, 64, max_new, 1 << 40) == UNSUPPORTED
        assert "pairs" in vq3.lib.vq3_last_error().decode()


def test_binding_makes_the_larger_workspace(world, monkeypatch):  # noqa: F811
    sizes = {0: 5 << 20, 4: 1 << 20}
    monkeypatch.setattr(vq3.lib, "vq3_attention_workspace_bytes", lambda h, k, d, n: sizes[n])
    world.answers = [-5]
    run_paged()
    assert [c[3][-2] for c in world.calls] == [1 << 20, 5 << 20]
    # a caller's own is the caller's to size, and other refusals are not tried again
    for answer, kw in ((-5, dict(ws=Tensor((1 << 20,), torch.uint8))), (-3, {})):
        world.answers, n = [answer], len(world.calls)
        with pytest.raises(vq3.Vq3Error):
            run_paged(**kw)
        assert len(world.calls) == n + 1


@pytest.mark.parametrize("kv_heads", [(1 << 16) + 1, 1 << 20])
def test_no_workspace_size_for_what_the_calls_refuse(kv_heads):
    assert vq3.attention_workspace_bytes(1 << 16, 1 << 16, 64) > 0
    assert vq3.attention_workspace_bytes(kv_heads, kv_heads, 64) == 0
